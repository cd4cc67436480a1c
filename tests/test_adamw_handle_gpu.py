"""What a DoraAdamW handle keeps for itself: its step's workspace, and its state when a load is refused."""
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()


def handle(bits=8, sizes=(3000, 500)):
    gen = torch.Generator(device="cuda").manual_seed(sum(sizes))
    params, grads = ([torch.randn(n, generator=gen, device="cuda").to(BF) for n in sizes] for _ in range(2))
    return params, grads, dw.DoraAdamW(params, grads, lr=1e-2, state_bits=bits, master=True)


def test_a_norm_on_the_side_leaves_the_steps_workspace():
    """grad_norm may run on another stream, or in another graph, while a step is between its two kernels."""
    _, grads, opt = handle()
    want, _ = dw.dora_grad_norm(grads, 0.5)
    opt._ws.fill_(7)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    norms = [opt.grad_norm(0.5)[0], opt.grad_norm(0.5, stream=st)[0]]
    torch.cuda.synchronize()
    assert (opt._ws == 7).all()
    assert all(torch.equal(n, want) for n in norms)
