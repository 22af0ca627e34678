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


BAD_FLAGS = [dict(dtype=torch.int64), dict(dtype=torch.float32), dict(dtype=torch.int32, device="cpu"),
             dict(dtype=torch.int32, n=0)]


@pytest.mark.parametrize("bad", BAD_FLAGS)
def test_flag_refusals_on_the_host(K, bad):
    """The kernels write to the flag through its address, so its type and device are checked before a launch."""
    from host_memory_streamed_stream_gb300 import MTError

    dev = torch.device("meta")
    with pytest.raises(MTError, match="err"):
        K._err(torch.zeros(bad.get("n", 1), dtype=bad["dtype"], device=bad.get("device", dev)), dev)
    good = torch.zeros(1, dtype=torch.int32, device=dev)
    assert K._err(good, dev) is good


@pytest.mark.gpu
@pytest.mark.parametrize("bad", BAD_FLAGS)
def test_flag_refusals(K, bad):
    from host_memory_streamed_stream_gb300 import MTError

    err = torch.zeros(bad.get("n", 1), dtype=bad["dtype"], device=bad.get("device", "cuda"))
    x = torch.zeros(8, 6 * 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    tab = K.rotary_table(K.rotary_inv_freq(64), 8)
    q, k, v = x[:, :256], x[:, 256:320], x[:, 320:]
    o, lse = K.attn_span_fwd(q, k, v, 1, 8, 4, 1, 64)
    _, rstd = K.qk_norm_rope(x, g, g, 4, 1, 64, tab)
    for call in (lambda: K.rotary(x, 5, 64, tab, err=err), lambda: K.qk_norm_rope(x, g, g, 4, 1, 64, tab, err=err),
                 lambda: K.qk_norm_rope_bwd(x, x, g, g, rstd, 4, 1, 64, tab, err=err),
                 lambda: K.attn_span_fwd(q, k, v, 1, 8, 4, 1, 64, err=err),
                 lambda: K.attn_span_bwd(q, k, v, o, lse, o, 1, 8, 4, 1, 64, err=err),
                 lambda: K.attn_fwd(x, 1, 8, 4, 1, 64, err=err),
                 lambda: K.gemm(x, False, x, False, 8, 8, 384, err=err)):
        with pytest.raises(MTError, match="err"):
            call()


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
