"""GPU checks of the q/k norm at the edges of what its header and binding allow."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    from rl_train_numerics_b200 import _abi
    return _abi


def draw(T, Hq, Hk, d, seed, dt=BF, gdt=F32):
    r = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    return (rand(T, Hq, d).to(dt).cuda(), rand(T, Hk, d).to(dt).cuda(),
            rand(T, Hq, d).to(gdt).cuda(), rand(T, Hk, d).to(gdt).cuda(),
            (1 + 0.3 * rand(d)).cuda(), (1 + 0.3 * rand(d)).cuda())


@pytest.mark.parametrize("have", [(), ("dq",), ("dk", "dwk"), ("dwq",)])
def test_gradient_buffers_that_are_not_given_are_made(gdn, have):
    q, k, doq, dok, wq, wk = draw(9, 4, 2, 64, 3)
    kw = dict(norm="rms", wq=wq, wk=wk)
    want = gdn.qk_norm_backward(q, k, doq, dok, **kw)
    buf = {s: torch.empty_like(want[s]) for s in have}
    got = gdn.qk_norm_backward(q, k, doq, dok, grads=buf, **kw)
    assert set(got) == set(want) and all(got[s] is buf[s] for s in have)
    assert all(torch.equal(got[s], want[s]) for s in want)
