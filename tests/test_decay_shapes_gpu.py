"""gdn_decay_step and gdn_decay_prefill over every d_k, both types, and rows
that can and cannot be read in wide pieces, against the rule in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests import serving_ref as ref  # noqa: E402
from tests.test_decay_gpu import _near, _run_window, _window  # noqa: E402
from tests.test_decay_wide_gpu import LONG, Prompt, assert_wide, segments  # noqa: E402


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("d_v", [36, 128, 33, 50])       # the last two entry by entry
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d_k", [16, 32, 64, 128])
def test_windows(d_k, kind, d_v, per_head):
    layers, t_lane, h_v, h_k, T = 2, [5, 0, 1, 8], 6, 2, 8
    x = _window(layers, t_lane, h_v, h_k, d_k, d_v, T, kind, "slow", per_head)
    o, S = _run_window(x, t_lane, per_head)
    kept, S0 = _run_window(x, t_lane, per_head, keep=True)
    assert torch.equal(kept, o) and torch.equal(S0, x["S"])
    assert torch.equal(_run_window(x, t_lane, per_head, want_o=False)[1], S)
    for y in range(layers):
        for n, m in enumerate(t_lane):
            assert (o[y, n, m:] == 7).all()
            if m == 0:
                assert torch.equal(S[y, n], x["S"][y, n])
                continue
            rep = lambda z: z[y, n, :m].double().repeat_interleave(h_v // h_k, 1)
            g = x["g"][y].expand(m, h_v) if per_head else x["g"][y, n, :m]
            wo, wS, mo, mS = ref.decay_chain(rep(x["q"]), rep(x["k"]), x["v"][y, n, :m], g,
                                             x["S"][y, n], 0.5)
            _near(o[y, n, :m], wo, mo, ref.step_bound(d_k, m), "o layer %d lane %d" % (y, n))
            _near(S[y, n], wS, mS, ref.step_bound(d_k, m), "S layer %d lane %d" % (y, n))


@pytest.mark.parametrize("d_v", [48, 50, 61])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d_k", [16, 32, 64, 128])
def test_prompts_of_few_workgroups(d_k, kind, d_v):
    lens = [700, 0, 65, 1]
    assert segments(lens, 4, 2, d_k, d_v) == 6 + 3
    x = Prompt(lens, 4, 2, d_k, d_v, kind)
    o, S = x.run()
    assert torch.equal(x.run(want_o=False)[1], S)
    x.check(o, S)


@pytest.mark.parametrize("d_v", [96, 99])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d_k", [32, 64, 128])
def test_prompts_of_many_workgroups(d_k, kind, d_v):
    assert assert_wide(LONG, 32, 8, d_k, d_v) > len(LONG)
    x = Prompt(LONG, 32, 8, d_k, d_v, kind)
    o, S = x.run()
    assert torch.equal(x.run(want_o=False)[1], S)
    x.check(o, S)
