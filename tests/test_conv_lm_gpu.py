"""The example model's step: its gradients against torch's in fp32, and that it learns."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_gradients_match_autograd():
    """Activations and their gradients pass through bf16 (2^-9 each way, four roundings a layer): within 3%."""
    import torch.nn.functional as F

    from examples.conv_lm_step import ConvLM, batch_of
    from implicit_gemm_gb300 import build
    build.build()
    model = ConvLM(vocab=64)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    tokens, targets = batch_of(gen, 16, 128, 64)
    loss = model.gradients(tokens, targets)
    table = model.table.clone().requires_grad_()
    ws = [layer.w.float().requires_grad_() for layer in model.layers]
    h = table[tokens] * model.scale
    for w in ws:
        u = F.pad(h.mT, (w.shape[2] - 1, 0))
        h = h + F.gelu(F.conv1d(u, w[0].permute(0, 2, 1)).mT)
    ref = F.cross_entropy((h.reshape(-1, model.channels) @ table.t()), targets.reshape(-1))
    ref.backward()
    assert abs(float(loss) - float(ref.detach())) < 0.02 * float(ref.detach())
    far = lambda a, b: float((a.float() - b).norm() / b.norm())  # noqa: E731
    assert far(model.dtable, table.grad) < 0.03
    for layer, w in zip(model.layers, ws):
        assert far(layer.dw, w.grad) < 0.03


def test_learns():
    from examples.conv_lm_step import main
    losses = main(60, say=lambda *_: None)
    assert losses[-1] < 0.5 * losses[0]
