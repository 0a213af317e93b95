"""Embedding rows and their gradient against the definition in 64 bits, on the
GPU: sizes around the sort's, tiles' and lanes' borders, every pair of formats,
views at odd offsets and row strides, tokens without a row, padding, runs that
cross tiles, empty calls, infinities, tables past 2^31 elements, streams and
captured graphs."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
# half a step relative to the value, and half the smallest number
HALF = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"fp32": 2.0 ** -150, "fp16": 2.0 ** -25, "bf16": 2.0 ** -134}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def view(shape, dtype, shift, g=None, fill=None):
    """A contiguous tensor `shift` elements into a buffer with a border of 64
    elements on either side, and that buffer."""
    n = math.prod(shape)
    buf = torch.full((n + 64 + 64 + shift,), 7.0, dtype=dtype, device="cuda")
    t = buf[64 + shift:64 + shift + n].view(shape)
    if g is not None:
        t.copy_(torch.randn(shape, generator=g, device="cuda"))
    elif fill is not None:
        t.fill_(fill)
    return t, buf


def border_kept(buf, n, shift):
    keep = torch.cat((buf[:64 + shift], buf[64 + shift + n:]))
    assert bool((keep == 7.0).all()), "memory beside the output was written"


def assert_near(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    bad &= ~(torch.isinf(want) & (got.double() == want))
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:4], want[bad][:4])


LOOKUPS = [  # tokens, vocab, dim, table, out, shift, wide
    (1, 5, 1, "bf16", "bf16", 0, True), (1, 32000, 4096, "bf16", "bf16", 0, True),
    (7, 9, 7, "fp16", "fp32", 1, False), (65, 100, 8, "fp32", "fp16", 3, True),
    (300, 1000, 9, "bf16", "fp16", 5, True), (1025, 50, 61, "fp32", "fp32", 1, False),
    (513, 77, 1023, "fp16", "bf16", 7, True), (64, 3, 2048, "bf16", "fp32", 2, True),
    (0, 4, 16, "bf16", "bf16", 0, True), (5, 0, 16, "fp32", "bf16", 0, True),
    (6, 4, 0, "fp32", "bf16", 0, True)]


@pytest.mark.parametrize("n,vocab,dim,table,out,shift,wide", LOOKUPS)
def test_lookup(zf, n, vocab, dim, table, out, shift, wide):
    g = gen(n + dim)
    w, _ = view((vocab, dim), DT[table], shift, g)
    tok = torch.randint(-2, vocab + 3, (n,), generator=g, device="cuda") + 11
    tok = tok if wide else tok.int()
    y, buf = view((n, dim), DT[out], shift)
    scale = float(np.float32(math.sqrt(dim + 1)))
    zf.zero_embed_lookup(tok, w, y, scale=scale, first=11)
    row = tok.long() - 11
    ok = (row >= 0) & (row < vocab)
    want = torch.zeros(n, dim, dtype=torch.float64, device="cuda")
    want[ok] = w[row[ok]].double() * scale
    # the product's rounding in fp32, then the output's
    half = 0.0 if out == "fp32" else HALF[out]
    assert_near(y, want, want.abs() * (U + half * (1 + U)) + LEAST[out])
    border_kept(buf, n * dim, shift)


def test_lookup_into_columns_of_a_wider_buffer(zf):
    g = gen(5)
    w = torch.randn(40, 24, generator=g, device="cuda").bfloat16()
    tok = torch.randint(0, 40, (30,), generator=g, device="cuda")
    wide = torch.full((30, 100), 7.0, dtype=torch.bfloat16, device="cuda")
    zf.zero_embed_lookup(tok, w, wide[:, 33:57], scale=1.0)
    assert torch.equal(wide[:, 33:57], w[tok])
    assert bool((wide[:, :33] == 7).all()) and bool((wide[:, 57:] == 7).all())
    # tokens of any shape, an output with the same leading dimensions
    y = torch.empty(5, 6, 24, dtype=torch.bfloat16, device="cuda")
    zf.zero_embed_lookup(tok.view(5, 6), w, y)
    assert torch.equal(y, w[tok].view(5, 6, 24))


@pytest.mark.parametrize("n_slots,slot,offset,vocab,dim,shift", [
    (1, 4096, 0, 64, 64, 0), (4, 1000, 17, 60, 61, 1), (8, 257, 3, 33, 62, 3), (3, 256, 0, 12, 64, 0),
    (64, 8, 0, 8, 64, 0), (7, 5, 1, 2, 17, 0), (2, 100000, 1000, 195, 1016, 0), (5, 776, 8, 60, 64, 4)])
def test_lookup_in_the_int8_payload(zf, n_slots, slot, offset, vocab, dim, shift):
    g = gen(slot)
    nb = -(-slot // 256)
    q = torch.randint(-127, 128, (n_slots * slot + shift,), generator=g, device="cuda", dtype=torch.int8)[shift:]
    s = torch.rand(n_slots * nb, generator=g, device="cuda") + 0.1
    assert offset + vocab * dim <= n_slots * slot
    tok = torch.randint(0, vocab + 1, (2 * vocab + 3,), generator=g, device="cuda")
    tok[0], tok[1] = vocab - 1, 0
    scale = float(np.float32(1.7))
    e = torch.arange(vocab * dim, device="cuda") + offset
    scales = s[e // slot * nb + e % slot // 256].double()
    full = (q[e].double() * scales * scale).view(vocab, dim)
    for out in ("fp32", "bf16"):
        y, buf = view((tok.numel(), dim), DT[out], shift)
        zf.zero_embed_lookup_int8(tok, q, s, n_slots, slot, offset, vocab, y, scale=scale)
        want = torch.cat((full, torch.zeros(1, dim, dtype=torch.float64, device="cuda")))[tok]
        # two fp32 products, then the output's rounding
        half = 0.0 if out == "fp32" else HALF[out]
        assert_near(y, want, want.abs() * (2.01 * U + half * (1 + 3 * U)) + LEAST[out])
        border_kept(buf, tok.numel() * dim, shift)


def test_lookup_agrees_with_the_restored_payload(zf):
    """The gathered payload restored whole and the rows read straight from it."""
    g = gen(9)
    slot, n_slots, vocab, dim = 5000, 6, 400, 72
    q = torch.randint(-127, 128, (n_slots * slot,), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(n_slots * 20, generator=g, device="cuda")
    flat = torch.empty(n_slots * slot, device="cuda")
    zf.zero_dequant_allgather(q, s, n_slots, slot, flat)
    tok = torch.randint(0, vocab, (1000,), generator=g, device="cuda")
    a, b = torch.empty(1000, dim, device="cuda"), torch.empty(1000, dim, device="cuda")
    zf.zero_embed_lookup_int8(tok, q, s, n_slots, slot, 123, vocab, a)
    zf.zero_embed_lookup(tok, flat[123:123 + vocab * dim].view(vocab, dim), b)
    assert torch.equal(a, b)


def reference(tok, dy, vocab, scale, first=0, padding=None, old=None):
    """(gradient, bound of the fp32 sums' error without the output's rounding), 64 bits."""
    row = tok.long().view(-1) - first
    ok = (row >= 0) & (row < vocab)
    if padding is not None:
        ok &= tok.view(-1) != padding
    d = dy.reshape(row.numel(), dy.shape[-1]).double()[ok]
    z = torch.zeros(vocab, d.shape[1], dtype=torch.float64, device="cuda")
    total, size = z.clone().index_add_(0, row[ok], d), z.clone().index_add_(0, row[ok], d.abs())
    count = torch.bincount(row[ok], minlength=vocab).double()[:, None]
    y = total * scale
    # count - 1 additions in any order, each partial sum at most `size`; the
    # product with the scale; the addition to the old value
    tol = scale * size * U * (count + 1) * 1.001
    if old is not None:
        y = y + old.double()
        tol = tol + (y.abs() + tol) * U
    return y, tol


GRADS = [  # tokens, vocab, dim, dy, grad, accumulate, shift, wide
    (1, 1, 1, "fp32", "fp32", False, 0, True), (1, 10, 8, "bf16", "bf16", True, 0, True),
    (7, 3, 9, "fp16", "fp32", False, 1, False), (8, 300, 61, "bf16", "fp16", False, 3, True),
    (9, 5, 512, "fp32", "bf16", True, 0, True), (100, 255, 513, "bf16", "fp32", True, 5, True),
    (1000, 256, 40, "fp16", "fp16", False, 0, True), (1024, 257, 7, "fp32", "fp32", True, 1, False),
    (4095, 1000, 16, "bf16", "bf16", False, 0, True), (4096, 65535, 8, "bf16", "fp32", False, 0, True),
    (4097, 65536, 8, "bf16", "fp32", False, 1, True), (5000, 2, 33, "fp32", "fp32", True, 0, True),
    (30011, 50021, 24, "bf16", "fp32", True, 1, True), (20000, 300000, 8, "fp16", "bf16", False, 0, True),
    (131072, 777, 8, "bf16", "fp32", False, 0, True), (131073, 70000, 8, "bf16", "fp16", True, 0, False),
    # either side of where the sort begins: tokens, and tokens by columns
    (2048, 300, 24, "bf16", "bf16", False, 1, True), (2049, 300, 24, "bf16", "bf16", False, 1, True),
    (600, 50, 4100, "bf16", "fp32", True, 0, True), (700, 50, 4100, "fp16", "fp16", False, 3, True),
    (1024, 400, 1030, "fp32", "bf16", False, 0, True), (2048, 5, 3, "fp32", "fp32", True, 1, False),
    (2100, 5, 3, "fp16", "fp32", False, 1, False), (300, 17, 8, "bf16", "bf16", True, 1, True),
    (70000, 1, 5, "fp32", "fp32", False, 0, True), (0, 50, 16, "bf16", "bf16", False, 0, True),
    (0, 50, 16, "bf16", "bf16", True, 0, True), (9, 0, 16, "bf16", "bf16", False, 0, True),
    (9, 5, 0, "bf16", "bf16", False, 0, True)]


@pytest.mark.parametrize("n,vocab,dim,dyt,gt,accumulate,shift,wide", GRADS)
def test_grad(zf, n, vocab, dim, dyt, gt, accumulate, shift, wide):
    g = gen(n + 31 * dim)
    dy, _ = view((n, dim), DT[dyt], shift, g)
    # half of the tokens by rank (frequent ones fill tiles), half even; some outside
    tok = torch.randint(-1, vocab + 2, (n,), generator=g, device="cuda")
    often = (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(max(vocab, 1) + 1)).exp()
    tok[::2] = often.long()[::2] - 1
    tok = (tok + 6) if wide else (tok + 6).int()
    padding = 6 + vocab // 2
    grad, buf = view((vocab, dim), DT[gt], shift, g if accumulate else None)
    old = grad.clone() if accumulate else None
    scale = float(np.float32(0.37))
    zf.zero_embed_grad(tok, dy, grad, scale=scale, first=6, padding=padding, accumulate=accumulate)
    want, tol = reference(tok, dy, vocab, scale, 6, padding, old)
    half = 0.0 if gt == "fp32" else HALF[gt]
    assert_near(grad, want, tol + (want.abs() + tol) * half + LEAST[gt])
    border_kept(buf, vocab * dim, shift)
    if accumulate and vocab:
        row = tok.long() - 6
        hit = torch.zeros(vocab + 1, dtype=torch.bool, device="cuda")
        hit[torch.where((row >= 0) & (row < vocab) & (tok != padding), row, vocab)] = True
        assert torch.equal(grad[~hit[:-1]], old[~hit[:-1]])


@pytest.mark.parametrize("n,vocab,dim", [(500, 3, 40), (2000, 40, 24), (3000, 40, 24), (4096, 4096, 8), (50000, 3000, 17),
                                         (200000, 60000, 9), (70000, 300, 1500)])
@pytest.mark.parametrize("accumulate", (False, True))
def test_grad_of_whole_numbers_is_exact(zf, n, vocab, dim, accumulate):
    """Whole numbers whose sums fp32 holds: every order of adding gives the same,
    so that a row lost, doubled or added elsewhere shows."""
    g = gen(n)
    tok = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    tok[n // 3:n // 2] = vocab - 1
    dy = torch.randint(-8, 9, (n, dim), generator=g, device="cuda").float()
    grad = torch.randint(-8, 9, (vocab, dim), generator=g, device="cuda").float()
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, tok, dy.double())
    if accumulate:
        want += grad.double()
    again = grad.clone()
    zf.zero_embed_grad(tok, dy, grad, accumulate=accumulate)
    assert torch.equal(grad.double(), want)
    zf.zero_embed_grad(tok, dy.bfloat16(), again, accumulate=accumulate)
    assert torch.equal(again.double(), want)


def test_grad_is_the_same_every_time_and_on_its_own_workspace(zf):
    g = gen(3)
    tok = torch.randint(0, 500, (40000,), generator=g, device="cuda")
    dy = torch.randn(40000, 48, generator=g, device="cuda")
    a, b = torch.empty(500, 48, device="cuda"), torch.empty(500, 48, device="cuda")
    need = zf.zero_embed_grad_workspace(40000, 500, 48)
    buf = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    zf.zero_embed_grad(tok, dy, a)
    zf.zero_embed_grad(tok, dy, b, workspace=buf[:need])
    assert torch.equal(a, b)
    assert bool((buf[need:] == 0xAB).all()), "the workspace's end was passed"


def test_grad_of_strided_and_broadcast_rows(zf):
    g = gen(4)
    tok = torch.randint(0, 30, (200,), generator=g, device="cuda")
    wide = torch.randn(200, 70, generator=g, device="cuda")
    a, b = torch.empty(30, 33, device="cuda"), torch.empty(30, 33, device="cuda")
    zf.zero_embed_grad(tok, wide[:, 9:42], a)
    zf.zero_embed_grad(tok, wide[:, 9:42].contiguous(), b)
    assert torch.equal(a, b)
    row = torch.randint(-8, 9, (33,), generator=g, device="cuda").float()
    zf.zero_embed_grad(tok, row.expand(200, 33), a)           # one row for every token
    want = torch.bincount(tok, minlength=30).float()[:, None] * row
    assert torch.equal(a, want)


def test_grad_keeps_infinities_to_their_rows(zf):
    tok = torch.tensor([3, 1, 3, 2, 9], device="cuda")
    dy = torch.ones(5, 16, device="cuda")
    dy[0, 2], dy[1, 3], dy[4, 4] = math.inf, math.nan, math.nan
    grad = torch.empty(5, 16, device="cuda")
    zf.zero_embed_grad(tok, dy, grad)                         # token 9 has no row here
    want = torch.zeros(5, 16, device="cuda")
    want[1], want[2], want[3] = 1, 1, 2
    want[3, 2], want[1, 3] = math.inf, math.nan
    assert torch.equal(torch.nan_to_num(grad, nan=-7.0), torch.nan_to_num(want, nan=-7.0))


def test_grad_against_differences(zf):
    """<dy, lookup(W + h D) - lookup(W)> / h = <grad, D>, on whole numbers: exactly."""
    g = gen(6)
    w = torch.randint(-9, 10, (50, 12), generator=g, device="cuda").float()
    d = torch.randint(-3, 4, (50, 12), generator=g, device="cuda").float()
    tok = torch.randint(-2, 53, (333,), generator=g, device="cuda")
    dy = torch.randint(-3, 4, (333, 12), generator=g, device="cuda").float()
    y0, y1, grad = torch.empty(333, 12, device="cuda"), torch.empty(333, 12, device="cuda"), torch.empty_like(w)
    zf.zero_embed_lookup(tok, w, y0, scale=2.0)
    zf.zero_embed_lookup(tok, w + d, y1, scale=2.0)
    zf.zero_embed_grad(tok, dy, grad, scale=2.0)
    assert float((dy.double() * (y1 - y0).double()).sum()) == float((grad.double() * d.double()).sum())


def test_tables_past_2_to_the_31_elements(zf):
    vocab, dim = 300000, 8192
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    rows = [vocab - 1, 262143, 262144, 131071, 0]
    for k, r in enumerate(rows):
        w[r] = k + 1.0
    tok = torch.tensor(rows + [5], device="cuda")
    y = torch.empty(6, dim, dtype=torch.bfloat16, device="cuda")
    zf.zero_embed_lookup(tok, w, y)
    assert torch.equal(y[:, 0].float().cpu(), torch.tensor([1., 2, 3, 4, 5, 0]))
    assert bool((y == y[:, :1]).all())
    w.fill_(9.0)
    zf.zero_embed_grad(tok, y, w)                             # every row written
    assert torch.equal(w[tok], y)
    assert float(w.abs().sum(dtype=torch.float64)) == 15.0 * dim
    zf.zero_embed_grad(tok, y, w, accumulate=True)
    assert torch.equal(w[tok], 2 * y)


def test_on_another_stream(zf):
    g = gen(8)
    tok = torch.randint(0, 900, (9000,), generator=g, device="cuda")
    dy = torch.randn(9000, 32, generator=g, device="cuda")
    a, b = torch.empty(900, 32, device="cuda"), torch.empty(900, 32, device="cuda")
    zf.zero_embed_grad(tok, dy, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        b.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        zf.zero_embed_grad(tok, dy, b, stream=s)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, b)


def test_captured_calls_replay_as_eager_ones(zf):
    g = gen(10)
    n, vocab, dim = 6000, 700, 40
    w = torch.randn(vocab, dim, generator=g, device="cuda").bfloat16()
    tok = torch.zeros(n, dtype=torch.int64, device="cuda")
    dy = torch.zeros(n, dim, device="cuda")
    y, grad = torch.empty(n, dim, device="cuda"), torch.zeros(vocab, dim, device="cuda")
    zf.zero_embed_lookup(tok, w, y)
    zf.zero_embed_grad(tok, dy, grad)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zf.zero_embed_lookup(tok, w, y)
        zf.zero_embed_grad(tok, dy, grad)
    for k in range(3):
        tok.copy_(torch.randint(0, vocab, (n,), generator=g, device="cuda"))
        dy.copy_(torch.randn(n, dim, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        y2, grad2 = torch.empty_like(y), torch.empty_like(grad)
        zf.zero_embed_lookup(tok, w, y2)
        zf.zero_embed_grad(tok, dy, grad2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(grad, grad2), k


@pytest.mark.parametrize("dim", [1, 3, 7, 8, 13, 33, 130])
@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 700, 5000])
def test_rows_without_a_token_are_zeros(zf, n, gt, dim):
    """Many rows to a block, at every offset of the first one; what lies around stays."""
    vocab = 70001
    tok = torch.randint(0, vocab, (n,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    tok[-1], tok[0] = vocab - 1, 0
    dy = torch.ones(n, dim, device="cuda")
    want = torch.bincount(tok, minlength=vocab).to(gt)[:, None].expand(vocab, dim)
    for shift in (0, 1, 2, 3, 5, 7):
        b = torch.full((vocab * dim + 16,), 9.0, dtype=gt, device="cuda")
        g = b[shift:shift + vocab * dim].view(vocab, dim)
        zf.zero_embed_grad(tok, dy, g)
        assert torch.equal(g, want)
        assert bool((b[:shift] == 9.0).all()) and bool((b[shift + vocab * dim:] == 9.0).all())
