"""The mean error of the log-probabilities, which is what a sequence's sum adds up, against float64.

Tolerance. Rounding a result of size 2^e to fp32 is an error of 2^(e - 23) / sqrt(12) in the root mean square, and its
terms err by 1.5e-7 of their own, which a mean over T rows divides by sqrt(T). What does not average out is to stay
below 1e-8: the factor's two floats (2^-34 of numbers of size 30: 2e-9), the mean error of the power as known (1e-9)
and of the logarithm (at most 2^-25 a row, of either sign, 5e-9 in the mean). The bound is 1e-8 and 4.5 of the mean's
own deviations, which is below 5e-8: the power's mean error left in place would pass it, and so would a factor rounded
to one float (1e-7).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


@pytest.mark.parametrize("T,V", [(8000, 1001), (8000, 4001), (8000, 32000), (6000, 152064)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 1 / 0.7])
def test_mean_error(K, T, V, kind, scale):
    a = float(np.float32(scale))
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.zeros(T, (V + 7) // 8 * 8, dtype=TYPES[kind], device="cuda")[:, :V]
    for rows in range(0, T, 500):
        z[rows:rows + 500] = 2.0 * torch.randn(min(500, T - rows), V, device="cuda", generator=g)
    lab = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    logp, lse = K.token_logprobs(z, lab, scale=a)
    flat = torch.full((T,), -15.0, device="cuda")
    lp = K.policy_loss(z, lab, flat, torch.ones(T, device="cuda"), scale=a)[2]
    want = torch.cat([torch.logsumexp(y.double() * a, 1) for y in z.split(200)])
    label = z[torch.arange(T, device="cuda"), lab.long()].double() * a
    for got, ref in ((logp, label - want), (lp, label - want), (lse, want)):
        step = 2.0 ** (ref.abs().log2().floor() - 23)
        bound = 1e-8 + 4.5 * float((step.square() / 12 + 1.5e-7 ** 2).mean().sqrt()) / T ** 0.5
        assert bound < 5e-8
        assert abs(float((got.double() - ref).mean())) <= bound
