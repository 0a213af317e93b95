"""The master tensors that a TensorListOptimizer is made from."""
import pytest
import torch

from test_gpu_multi_list import HP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_masters_that_require_gradients(zf, bits):
    """A model's own parameters as masters are copied, not recorded: the arenas
    are plain tensors that can be loaded, read and viewed."""
    torch.manual_seed(0)
    params = [torch.nn.Parameter(torch.randn(s, device="cuda")) for s in ((3, 100), (256,), (5,))]
    opt = zf.TensorListOptimizer(params, HP, state_bits=bits, loss_scale=1.0,
                                 grad_dtype=torch.float32, param_dtype=None)
    assert not opt.master.requires_grad and opt.master.grad_fn is None
    for v, p in zip(opt.views(opt.master), params):
        assert not v.requires_grad
        assert torch.equal(v, p.detach().view(-1))
    opt.bind([torch.randn_like(p).detach() for p in params])
    opt.step()
    saved = opt.master.clone()
    assert saved.cpu().numpy().shape == (4 * 256,)
    opt.master.copy_(saved)
    assert opt.master.grad_fn is None
    # the parameters are not the arena's: training state stays where it was
    assert all(p.requires_grad and p.grad is None for p in params)
