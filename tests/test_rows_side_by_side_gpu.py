"""Inputs and outputs that lie beside each other in the rows of one buffer share no element: they are taken and give
what they give in buffers of their own. Rows that do share elements are refused."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def _randn(*shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))


@pytest.mark.parametrize("T,h", [(50, 264), (2000, 4096), (1, 64)])
@pytest.mark.parametrize("first", ["x", "y"])
def test_layernorm_output_beside_its_input(K, T, h, first):
    gamma = torch.ones(h, dtype=torch.bfloat16, device="cuda")
    buf = torch.zeros(T, 2 * h + 8, dtype=torch.bfloat16, device="cuda")
    a, b = buf[:, :h], buf[:, h + 8:]
    x, y = (a, b) if first == "x" else (b, a)
    x.copy_(_randn(T, h))
    want = K.layernorm_fwd(x.clone(), gamma)
    got = K.layernorm_fwd(x, gamma, out=y)
    assert got[0] is y and all(torch.equal(p, q) for p, q in zip(got, want))
    assert torch.all(buf[:, h:h + 8] == 0)


@pytest.mark.parametrize("V", [1021, 9001, 40003])
def test_gradient_beside_the_logits(K, V):
    T, w = 70, (V + 7) // 8 * 8
    buf = torch.full((T, 2 * w), 5.0, dtype=torch.bfloat16, device="cuda")
    z, d = buf[:, :V], buf[:, w:w + V]
    z.copy_(2 * _randn(T, V))
    lab = (torch.arange(T, device="cuda") * 11 % V - 5).to(torch.int32)
    one, old = torch.ones(T, device="cuda"), torch.full((T,), -8.0, device="cuda")
    logits = torch.empty(T, w, dtype=torch.bfloat16, device="cuda")[:, :V]
    logits.copy_(z)
    _, lse = K.token_logprobs(logits, lab)
    want = K.token_logprobs_bwd(logits, lab, lse, one)
    K.token_logprobs_bwd(z, lab, lse, one, out=d)
    assert torch.equal(d, want) and torch.equal(z, logits)
    want = K.policy_loss(logits, lab, old, one)
    got = K.policy_loss(z, lab, old, one, out=d)
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(z, logits)
    assert torch.all(buf[:, V:w] == 5.0) and torch.all(buf[:, w + V:] == 5.0)


def test_shared_elements_are_refused(K):
    from host_memory_streamed_stream_gb300 import MTError

    T, h = 20, 64
    gamma = torch.ones(h, dtype=torch.bfloat16, device="cuda")
    buf = torch.zeros(T, 4 * h, dtype=torch.bfloat16, device="cuda")
    flat = buf.view(-1)
    x = buf[:, h:2 * h]
    lab, f = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, device="cuda")
    rows = torch.zeros(T, h, device="cuda")
    for out in (buf[:, h + 8:2 * h + 8], buf[:, h - 8:2 * h - 8], buf[:, h:2 * h],
                flat[h + 8:].as_strided((T - 1, h), (4 * h, 1)),  # a row less is another shape
                flat.as_strided((T, h), (2 * h, 1), 2 * h),       # another distance between rows
                flat.as_strided((T, h), (4 * h, 1), 2 * h - 8),
                flat.as_strided((T, h), (3 * h, 1), 0)):
        with pytest.raises(MTError):
            K.layernorm_fwd(x, gamma, out=out)
    # a row that ends in the next one's beginning
    wide = flat.as_strided((T, h + 8), (2 * h, 1), 0)
    with pytest.raises(MTError):
        K.token_logprobs_bwd(wide, lab, f, f, out=flat.as_strided((T, h + 8), (2 * h, 1), h))
    # fp32 logits and a bf16 gradient in the same bytes
    with pytest.raises(MTError):
        K.token_logprobs_bwd(rows, lab, f, f, out=rows.view(torch.bfloat16)[:, :h])
    with pytest.raises(MTError):
        K.token_logprobs_bwd(rows[:, :32], lab, f, f, out=rows.view(torch.bfloat16)[:, 56:88])
