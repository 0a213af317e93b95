"""Calls on a stream other than the current one, without a workspace, while the
current stream is still busy with memory of the same size that has been given
back: the call's own memory is not that."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


def busy_then_given_back(size):
    """Work on the current stream that ends with writes to memory already given back."""
    a = torch.ones(4096, 4096, device="cuda")
    for _ in range(30):
        a = a @ a * 2.0 ** -12
    t = torch.empty(size, dtype=torch.uint8, device="cuda")
    t.fill_(1)
    del t


def on_other_streams(size, call, result):
    """Compares a call on other streams, named as a user may, with one on its own."""
    call(None)
    torch.cuda.synchronize()
    want = result.clone()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for current, stream in ((torch.cuda.current_stream(), side), (torch.cuda.current_stream(), side.cuda_stream),
                            (other, side), (other, 0), (other, torch.cuda.default_stream())):
        result.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            busy_then_given_back(size)
            call(stream)
        torch.cuda.synchronize()
        assert torch.equal(result, want)


def test_embed_grad(zf):
    n, v, d = 9000, 900, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    tok = torch.randint(0, v, (n,), generator=g, device="cuda")
    dy, grad = torch.randn(n, d, generator=g, device="cuda"), torch.empty(v, d, device="cuda")
    size = zf.zero_embed_grad_workspace(n, v, d)
    assert size > 0
    on_other_streams(size, lambda s: zf.zero_embed_grad(tok, dy, grad, stream=s), grad)


def test_weight_grad(zf):
    g = torch.Generator(device="cuda").manual_seed(2)
    s, grad = zf.Saved8(4000, 300), torch.empty(200, 300, device="cuda")
    zf.zero_act_save8(torch.randn(4000, 300, generator=g, device="cuda"), s)
    dy = torch.randn(4000, 200, generator=g, device="cuda").bfloat16()
    size = zf.zero_weight_grad8_workspace(4000, 200, 300)
    assert size > 0
    on_other_streams(size, lambda st: zf.zero_weight_grad8(dy, s, grad, stream=st), grad)


def test_captured_on_a_forked_stream(zf):
    """A graph that forks: the call goes on the branch, its memory belongs to the graph."""
    n, v, d = 6000, 500, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    tok = torch.randint(0, v, (n,), generator=g, device="cuda")
    dy, grad, want = torch.randn(n, d, generator=g, device="cuda"), torch.empty(v, d, device="cuda"), torch.empty(v, d, device="cuda")
    zf.zero_embed_grad(tok, dy, grad)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        zf.zero_embed_grad(tok, dy, grad, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        dy.copy_(torch.randn(n, d, generator=g, device="cuda"))
        grad.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        zf.zero_embed_grad(tok, dy, want)
        torch.cuda.synchronize()
        assert torch.equal(grad, want)


def test_an_optimizers_first_step(zf):
    """The gradient shard that the first step takes."""
    n = 100000
    g = torch.Generator(device="cuda").manual_seed(4)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, max_grad_norm=1.0)
    bufs = [torch.randn(n, generator=g, device="cuda").bfloat16() for _ in range(2)]
    start = torch.randn(n, generator=g, device="cuda")

    def step(several, stream, busy):
        master, slot = start.clone(), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        opt = zf.MultiShardOptimizer([master], hp, loss_scale=1.0) if several else zf.ShardOptimizer(master, hp, loss_scale=1.0)
        torch.cuda.synchronize()
        if busy:
            busy_then_given_back(4 * n)
        if several:
            opt.step_from_rank_buffers([bufs], [0], [slot], [0], stream=stream)
        else:
            opt.step_from_rank_buffers(bufs, 0, slot, 0, stream=stream)
        torch.cuda.synchronize()
        return master, slot

    for several in (False, True):
        want = step(several, None, False)
        assert not torch.equal(want[0], start)
        for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
            got = step(several, stream, True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
