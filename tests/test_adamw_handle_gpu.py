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


def snapshot(opt):
    return {k: v.clone().view(torch.uint8) if v.element_size() == 1 else v.clone() for k, v in opt.state_dict().items()}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad,error", [
    (lambda s: {"step": 3, "avg": s["avg"], "nothing": s["sq"]}, KeyError),
    (lambda s: {"step": 3, "avg": s["avg"], "sq": s["sq"][1:]}, ValueError),
    (lambda s: {"avg": s["avg"], "sq": s["sq"].float().double()}, ValueError),
    (lambda s: {"avg": s["avg"], "step": -1}, ValueError)])
def test_a_refused_load_changes_nothing(bits, bad, error):
    _, _, a = handle(bits)
    a.step()
    state = {k: v.clone() for k, v in a.state_dict().items()}
    params, _, b = handle(bits)
    before, p0 = snapshot(b), [p.clone() for p in params]
    with pytest.raises(error):
        b.load_state_dict(bad(state))
    after = snapshot(b)
    assert all(torch.equal(before[k], after[k]) for k in before)
    b.load_state_dict(state)  # the whole of it loads, and steps go on from there
    assert int(b.state_dict()["step"]) == 1 and all(torch.equal(x, y) for x, y in zip(params, p0))
    b.step()
    assert int(b.state_dict()["step"]) == 2
