"""The policy loss's KL term at its end: a label that the policy cannot produce is infinitely far from a reference
that can."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


@pytest.mark.parametrize("V", [104, 5000, 40000])
def test_impossible_label(K, V):
    inf = float("inf")
    z = torch.zeros(4, V, device="cuda")
    z[0, 3] = -inf     # exp(ref - logp) - (ref - logp) - 1 grows beyond all bounds as logp goes to -inf
    z[1, 3] = -1.0e9   # exp overflows, the difference is finite: the same
    lab = torch.tensor([3, 3, 3, -1], dtype=torch.int32).cuda()
    flat = torch.full((4,), -5.0, device="cuda")
    ref = torch.tensor([-5.0, -5.0, -inf, -5.0], device="cuda")  # and a reference that cannot: a term of +inf too
    loss, row, logp, _ = K.policy_loss(z, lab, flat, torch.ones(4, device="cuda"), ref_logp=ref, kl=0.1)
    assert logp[:2].tolist() == [-inf, -1.0e9]
    assert row.tolist() == [inf, inf, inf, 0.0] and float(loss) == inf
    # without the term: nothing to gain
    row = K.policy_loss(z, lab, flat, torch.ones(4, device="cuda"))[1]
    assert row[:2].tolist() == [0.0, 0.0]
