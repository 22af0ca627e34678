"""The device error flag that the kernel-level calls report to, and the README's example that reads it."""
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def test_check(K):
    from host_memory_streamed_stream_gb300 import MTError

    K.check(torch.zeros(1, dtype=torch.int32))
    for code, text in ((8, "position"), (5, "wait gave up")):
        with pytest.raises(MTError, match=text):
            K.check(torch.tensor([code], dtype=torch.int32))


def _example():
    """The README's attention block of packed documents."""
    with open(README) as f:
        blocks = [b.split("```")[0] for b in f.read().split("```python\n")[1:]]
    return next(b for b in blocks if "attn_span_bwd" in b)


@pytest.mark.gpu
def test_readme_example(K):
    """It runs, and a table that is too short for the documents does not pass unseen."""
    from host_memory_streamed_stream_gb300 import MTError

    rng = np.random.default_rng(3)

    def bf16(*shape):
        return torch.tensor(rng.standard_normal(shape), dtype=torch.float32).to(torch.bfloat16).cuda()

    given = dict(qkv=bf16(8192, 48 * 128), gq=bf16(128), gk=bf16(128), do=bf16(8192, 32 * 128))
    names = dict(given, qkv=given["qkv"].clone())
    exec(_example(), names)
    # 92 tokens after the last document are padding: no gradient; the others have one in every row
    d = names["dqkv"].float().abs().sum(1)
    assert bool((d[8100:] == 0).all()) and bool((d[:8100] > 0).all()) and bool(torch.isfinite(d).all())
    assert all(bool(torch.isfinite(names[n].float()).all()) for n in ("o", "dgq", "dgk"))
    short = _example().replace("high=4.0), s)", "high=4.0), 2048)")
    assert short != _example()
    with pytest.raises(MTError, match="position"):
        exec(short, dict(given, qkv=given["qkv"].clone()))
