"""The policy loss where it can go wrong by value or by the number of rows, on the GPU; formula, cases and tolerances
of test_gpu_policy.py."""
import numpy as np
import pytest

from test_gpu_policy import Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
lst = pytest.importorskip("layer_streamed_qlora_streaming_b200")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _result(c):
    torch.cuda.synchronize()
    assert lst.device_error() == 0
    return c.out[:4].cpu().numpy().copy(), c.logp[:c.T].cpu().numpy().copy(), c.dlog[:c.T * c.V].clone()


VOCABULARIES = [300, 5001, 40000, 310001]  # a warp, clusters, rows read twice


@pytest.mark.parametrize("V", VOCABULARIES)
def test_policy_zero_advantage_with_a_ratio_that_overflows(V):
    # u = 0 A = 0 whatever the ratio: all but the reported ratio is what any finite one gives
    c = Case(2, 4, V, "seq", 0.1, False, keep=1.1)
    c.adv[::3] = 0
    c.tadv.copy_(torch.from_numpy(c.adv))
    c.run()
    torch.cuda.synchronize()
    c.check()
    want = _result(c)
    c.told[::3] -= 200.0
    c.run()
    out, logp, dlog = _result(c)
    assert np.array_equal(out[:3], want[0][:3]) and np.isposinf(out[3])
    assert np.array_equal(logp, want[1]) and torch.equal(dlog, want[2])


@pytest.mark.parametrize("V", VOCABULARIES)
def test_policy_reference_without_a_weight_that_overflows(V):
    # kl_beta 0: the KL estimate is reported and nothing else depends on it
    c = Case(2, 4, V, "token", 0.0, True, keep=1.1)
    c.x[1, c.y[1]] = -np.inf  # a target that was ruled out: log-probability minus infinity
    c.tx.copy_(torch.from_numpy(c.x))
    c.run()
    want = _result(c)
    assert np.isneginf(want[1][1]) and np.all(np.isfinite(want[0])) and torch.all(torch.isfinite(want[2]))
    c.tref[5] += 500.0
    c.run(ref_logp=c.tref)
    out, logp, dlog = _result(c)
    assert np.array_equal(out[[0, 2, 3]], want[0][[0, 2, 3]]) and np.isposinf(out[1])
    assert np.array_equal(logp, want[1]) and torch.equal(dlog, want[2])
