"""gdn_draft_verify over vocabularies past 2^20."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests.test_draft_verify_gpu import _case, _check, _run  # noqa: E402


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("t_lane,V,pad,offset", [
    ([4, 0, 1, 2, 5, 3], (1 << 20) - 8192, 0, 0),      # about where the launches change
    ([4, 0, 1, 2, 5, 3], (1 << 20) - 8191, 0, 0),
    ([3, 2, 1, 4], (1 << 20) + 1, 7, 3),
    ([11, 1], 2222222, 1, 5),
])
def test_large_vocabularies(t_lane, V, pad, offset, kind, drafted):
    s = _case(t_lane, V, kind, drafted, pad=pad, offset=offset, right=0.6)
    _check(s, _run(s), 1.0)


@pytest.mark.parametrize("drafted", [False, True])
def test_rows_without_a_distribution(drafted):
    s = _case([3] * 6, (1 << 20) + 77, "f32", drafted)
    s["tokens"][:, 1] = 5
    s["uniforms"][:, 0] = 0.999
    s["logits"][0, 0, 9] = float("nan")
    s["logits"][1, 0, (1 << 20) + 76] = float("inf")
    s["logits"][2, 2] = -float("inf")
    s["it"][3] = 0.0
    s["tokens"][4, 1] = -1
    s["logits"][5, 0, 1 << 19:] = -float("inf")
    if drafted:
        s["draft"][5, 0, : 1 << 19] = -float("inf")
    _check(s, _run(s), 1.0)


def test_time_grows_as_the_vocabulary():
    """Four times the ids take about four times as long, where the draft falls
    and both rows count.  (Sixteen times is what a sum over all slices in every
    slice's workgroup takes.)"""
    times = []
    for V in (1 << 24, 1 << 26):
        x = torch.zeros(1, 2, V, device="cuda", dtype=torch.bfloat16)
        y = torch.zeros(1, 1, V, device="cuda", dtype=torch.bfloat16)
        y[..., : V // 2] = 1.0
        tokens = torch.full((1, 2), -1, device="cuda", dtype=torch.int32)
        u, it = torch.full((1, 2), 0.5, device="cuda"), torch.ones(1, device="cuda")
        m, token = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        ws = torch.empty(gdn.draft_verify_workspace_bytes(1, 2, V), dtype=torch.uint8, device="cuda")
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            gdn.draft_verify([2], x, y, tokens, u, it, m, token, ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        # p is flat, q is above it in the first half: half of the second half's ids
        assert m.item() == 1 and abs(token.item() - 3 * V // 4) <= 1
        print("2^%d ids: %.3f ms" % (V.bit_length() - 1, best), flush=True)
        times.append(best)
    assert times[1] <= 8 * times[0]


def test_captured_calls_over_a_large_vocabulary():
    """Replays on other rows, the workspace overwritten between them, against
    eager calls."""
    t_lane, V = [3, 0, 2], (1 << 20) + 5
    s = _case(t_lane, V, "bf16", True)
    m, token = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    accept = torch.zeros(3, 3, device="cuda")
    ws = torch.empty(gdn.draft_verify_workspace_bytes(3, 3, V), dtype=torch.uint8, device="cuda")

    def call():
        gdn.draft_verify(t_lane, s["logits"], s["draft"], s["tokens"], s["uniforms"], s["it"], m, token, ws,
                         accept=accept)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(5, 9):
        other = _case(t_lane, V, "bf16", True, seed=seed, right=0.5)
        for c in ("logits", "draft", "tokens", "uniforms", "it"):
            s[c].copy_(other[c])
        ws.fill_(seed)
        graph.replay()
        torch.cuda.synchronize()
        want = _run(s)
        for n in (0, 2):
            assert (m[n].item(), token[n].item()) == (want[0][n], want[1][n])
            assert torch.equal(accept[n, : t_lane[n] - 1].cpu().double(), want[2][n, : t_lane[n] - 1])
