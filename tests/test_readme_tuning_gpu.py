"""The README's fine-tuning examples: they run, and a token outside the vocabulary does not pass unseen."""
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _blocks():
    with open(README) as f:
        blocks = [b.split("```")[0] for b in f.read().split("```python\n")[1:]]
    return [next(b for b in blocks if name in b) for name in ("policy_loss", "preference_loss")]


def test_examples():
    from host_memory_streamed_stream_gb300 import MTError, _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels as K

    rng = np.random.default_rng(4)
    T, h, V = 256, 128, 1000

    def bf16(*shape, scale=1.0):
        return torch.tensor(rng.standard_normal(shape) * scale, dtype=torch.float32).bfloat16().cuda()

    def f32(a):
        return torch.tensor(a, dtype=torch.float32).cuda()

    def ids(n):
        return torch.tensor(rng.integers(0, n, T), dtype=torch.int32).cuda()

    names = dict(K=K, T=T, h=h, V=V, tok=ids(V), labels=ids(V), E=bf16(V, h, scale=0.1), W=bf16(V, h, scale=0.1),
                 gamma=bf16(h) * 0 + 1, beta=bf16(h), old_logp=f32(np.full(T, -7.0)), ref_logp=f32(np.full(T, -7.2)),
                 advantages=f32(rng.standard_normal(T)), weights=f32(np.full(T, 1 / T)),
                 bounds=torch.tensor([0, 60, 130, 200, 256], dtype=torch.int32).cuda(),
                 err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    names["labels"][:20] = -1
    policy, pairs = _blocks()
    exec(policy, names)
    used = torch.zeros(V, dtype=torch.bool, device="cuda")
    used[names["tok"].long()] = True
    for n in ("loss", "dgamma", "dbeta", "dW", "dE"):
        assert bool(torch.isfinite(names[n].float()).all()) and bool((names[n] != 0).any()), n
    assert bool((names["dE"][~used] == 0).all()) and bool((names["dz"][:20] == 0).all())
    exec(pairs, names)
    assert names["rewards"].shape == (4,) and bool(torch.isfinite(names["dz"].float()).all())
    names["tok"][5] = V
    with pytest.raises(MTError, match="token"):
        exec(policy, names)
