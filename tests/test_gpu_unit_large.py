"""A unit's operators at sizes that take branches of their own, on the GPU:
gradients whose zeros reach past what the sort's launches write, outputs that go
past the caches, more elements than one launch counts, row distances at and
above 2^25, and gradients of one row for all.  Whole numbers and comparisons with
small calls: every comparison is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, H, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def framed(shape, dtype, shift):
    """A contiguous tensor of sevens `shift` elements into a buffer of sevens with 64 more on
    either side, and a check that those stay."""
    n = shape[0] * shape[1]
    buf = torch.full((n + 128 + shift,), 7.0, dtype=dtype, device="cuda")

    def kept():
        assert bool((buf[:64 + shift] == 7.0).all()) and bool((buf[64 + shift + n:] == 7.0).all())
    return buf[64 + shift:64 + shift + n].view(shape), kept


def tokens_with_a_run(n, vocab, g):
    """Tokens all over the rows, the first and the last among them, one 200 times, some outside."""
    tok = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    tok[:200], tok[200], tok[201], tok[202], tok[203] = vocab // 2, 0, vocab - 1, -1, vocab
    return tok[torch.randperm(n, generator=g, device="cuda")]


# Each pass of the sort writes 80 MiB of zeros: two passes up to 65,535 rows, then three.  The
# sums' launch writes the others, from inside a row on where 40 MiB are no whole number of rows.
@pytest.mark.parametrize("n,vocab,dim,dtype,shift", [
    (6000, 40000, 3001, BF, 0), (6000, 40000, 3001, BF, 1), (5000, 60000, 2048, H, 0), (3000, 20000, 4099, F, 3),
    (70000, 9000, 6400, F, 0), (6000, 70001, 2003, F, 1), (4000, 140000, 1537, BF, 5), (3000, 30000, 1024, F, 0)])
def test_every_row_of_a_large_gradient(zf, n, vocab, dim, dtype, shift):
    g = gen(n + dim)
    tok = tokens_with_a_run(n, vocab, g)
    dy = torch.randint(-1, 2, (n, dim), generator=g, device="cuda").to(BF)
    row = torch.where((tok >= 0) & (tok < vocab), tok, vocab)
    # sums of at most some 200 units: exact in every type
    assert int(torch.bincount(row)[:vocab].max()) <= 256
    want = torch.zeros(vocab + 1, dim, device="cuda").index_add_(0, row, dy.float())[:vocab]
    grad, kept = framed((vocab, dim), dtype, shift)
    need = zf.zero_embed_grad_workspace(n, vocab, dim)
    assert need > 0
    # marks, counts and partial sums of an earlier use, all bits set
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    zf.zero_embed_grad(tok, dy, grad, workspace=ws)
    assert torch.equal(grad.float(), want)
    kept()
    # added to itself, in the same memory
    zf.zero_embed_grad(tok, dy, grad, accumulate=True, workspace=ws)
    assert torch.equal(grad.float(), 2 * want)
    kept()


def test_a_large_gradient_of_few_tokens(zf):
    for n, vocab, dim, dtype in ((3, 50000, 2501, BF), (600, 33000, 1999, F)):
        grad, kept = framed((vocab, dim), dtype, 1)
        g = gen(n)
        tok = torch.randint(0, vocab, (n,), generator=g, device="cuda")
        assert zf.zero_embed_grad_workspace(n, vocab, dim) == 0
        zf.zero_embed_grad(tok, torch.ones(n, dim, device="cuda"), grad)
        assert torch.equal(grad, torch.bincount(tok, minlength=vocab).to(dtype)[:, None].expand(vocab, dim))
        kept()


@pytest.mark.parametrize("table", [BF, H, F, torch.int8])
@pytest.mark.parametrize("out,n,dim,shift", [(BF, 70001, 1001, 1), (F, 40000, 1024, 0), (H, 9000, 8200, 4), (F, 33333, 1111, 3)])
def test_rows_of_128_mib_and_more(zf, table, out, n, dim, shift):
    g = gen(n)
    vocab = 5000
    tok = torch.randint(-1, vocab + 1, (n,), generator=g, device="cuda")
    y, kept = framed((n, dim), out, shift)
    assert y.nbytes >= 128 << 20
    if table == torch.int8:
        slot = vocab * dim + 77
        q = torch.randint(-127, 128, (slot,), generator=g, device="cuda", dtype=torch.int8)
        s = torch.rand(-(-slot // 256), generator=g, device="cuda")
        full = torch.empty(slot, device="cuda")
        zf.zero_dequant_allgather(q, s, 1, slot, full)
        w = full[13:13 + vocab * dim].view(vocab, dim)
        zf.zero_embed_lookup_int8(tok, q, s, 1, slot, 13, vocab, y)
    else:
        w = torch.randn(vocab, dim, generator=g, device="cuda").to(table)
        zf.zero_embed_lookup(tok, w, y)
    rows = torch.cat((w.to(out), torch.zeros(1, dim, dtype=out, device="cuda")))
    assert torch.equal(y, rows[torch.where((tok >= 0) & (tok < vocab), tok, vocab)])
    kept()


@pytest.mark.parametrize("kind", ("gelu", "gelu_tanh", "silu"))
@pytest.mark.parametrize("gated", (False, True))
@pytest.mark.parametrize("dtype,rows,cols,beside", [(BF, 33001, 2051, 3), (F, 17003, 2051, 5), (H, 40000, 2048, 0)])
def test_activations_of_128_mib_and_more(zf, dtype, rows, cols, beside, gated, kind):
    """The whole matrix, whose outputs go past the caches, against calls of 1000 rows, whose do not."""
    kind = {"gelu": zf.ZERO_GELU, "gelu_tanh": zf.ZERO_GELU_TANH, "silu": zf.ZERO_SILU}[kind]
    g = gen(rows)
    packed = torch.randn(rows, 2 * cols + beside, generator=g, device="cuda").to(dtype)
    x, u = packed[:, :cols], packed[:, cols + beside:] if gated else None
    y, kept = framed((rows, cols), dtype, 1)
    assert y.nbytes >= 128 << 20
    s, su = zf.Saved8(rows, cols), zf.Saved8(rows, cols) if gated else None
    zf.zero_act_forward8(kind, x, y, s, up=u, saved_up=su)
    kept()
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(dtype)
    both = torch.full((rows, 2 * cols + beside), 7.0, dtype=dtype, device="cuda")
    dx, dup = both[:, :cols], both[:, cols + beside:] if gated else None
    again = zf.Saved8(rows, cols)
    zf.zero_act_backward8(kind, dy, s, dx, saved_up=su, dup=dup, again=again)
    assert bool((both[:, cols:cols + beside] == 7.0).all())
    if not gated:
        assert bool((both[:, cols:] == 7.0).all())
    for r in range(0, rows, 1000):
        part, n = slice(r, min(rows, r + 1000)), min(rows, r + 1000) - r
        t, tu, ta = zf.Saved8(n, cols), zf.Saved8(n, cols) if gated else None, zf.Saved8(n, cols)
        ty, tx, td = torch.empty(n, cols, dtype=dtype, device="cuda"), torch.empty(n, cols, dtype=dtype, device="cuda"), None
        zf.zero_act_forward8(kind, x[part], ty, t, up=u[part] if gated else None, saved_up=tu)
        if gated:
            td = torch.empty(n, cols, dtype=dtype, device="cuda")
        zf.zero_act_backward8(kind, dy[part], t, tx, saved_up=tu, dup=td, again=ta)
        assert torch.equal(y[part], ty) and torch.equal(dx[part], tx)
        assert td is None or torch.equal(dup[part], td)
        for whole, small in ((s, t), (su, tu), (again, ta)):
            if whole is not None:
                assert torch.equal(whole.codes[part], small.codes) and torch.equal(whole.exponents[part], small.exponents)


@pytest.mark.parametrize("dtype,rows,cols", [(BF, 70000, 1001), (F, 33333, 1111)])
def test_restored_matrices_of_128_mib_and_more(zf, dtype, rows, cols):
    x = torch.randint(-64, 65, (rows, cols), generator=gen(rows), device="cuda").to(dtype)
    x[:, ::32] = 64.0                             # every block's unit is 1
    s = zf.Saved8(rows, cols)
    zf.zero_act_save8(x, s)
    y, kept = framed((rows, cols), dtype, 1)
    assert y.nbytes >= 128 << 20
    zf.zero_act_restore8(s, y)
    assert torch.equal(x, y)
    kept()


def test_more_rows_than_a_launch_counts(zf):
    """A checkpoint of 2^28 + 5 rows of one column: four groups of eight a row, and a launch counts 2^30."""
    rows = (1 << 28) + 5
    x = (torch.arange(rows, device="cuda", dtype=torch.int32) % 127 - 60).to(BF).view(rows, 1)
    s, y = zf.Saved8(rows, 1), torch.full((rows, 1), 7.0, dtype=BF, device="cuda")
    zf.zero_act_save8(x, s)
    zf.zero_act_restore8(s, y)
    assert torch.equal(x, y)                      # 7 bits: exact
    dx = torch.full((rows, 1), 7.0, dtype=BF, device="cuda")
    zf.zero_act_backward8(zf.ZERO_SILU, torch.ones(1, 1, dtype=BF, device="cuda").expand(rows, 1), s, dx)
    zf.zero_act_forward8(zf.ZERO_SILU, x, y, s)
    for got, call in ((y, lambda t, o: zf.zero_act_forward8(zf.ZERO_SILU, x[:127], o, t)),
                      (dx, lambda t, o: zf.zero_act_backward8(zf.ZERO_SILU, torch.ones(127, 1, dtype=BF, device="cuda"), t, o))):
        t, o = zf.Saved8(127, 1), torch.empty(127, 1, dtype=BF, device="cuda")
        zf.zero_act_save8(x[:127], t)
        call(t, o)
        whole = rows // 127 * 127
        assert bool((got[:whole].view(-1, 127) == o.view(1, 127)).all())
        assert torch.equal(got[whole:], o[:rows - whole])


def test_more_tokens_than_a_launch_counts(zf):
    """2^21 + 3 tokens of 512 groups each: a launch counts 2^30."""
    n, vocab, dim = (1 << 21) + 3, 1000, 4096
    w = torch.randn(vocab, dim, generator=gen(1), device="cuda").to(BF)
    for tok in (torch.arange(n, device="cuda") % vocab, torch.arange(n, device="cuda", dtype=torch.int32) % vocab):
        y = torch.full((n, dim), 7.0, dtype=BF, device="cuda")
        zf.zero_embed_lookup(tok, w, y)
        whole = n // vocab * vocab
        assert bool((y[:whole].view(-1, vocab, dim) == w).all()) and torch.equal(y[whole:], w[:n - whole])


# ------------------------------------------------------------------ weight gradients
def kept_input(zf, rows, cols, g):
    s = zf.Saved8(rows, cols)
    zf.zero_act_save8(torch.randn(rows, cols, generator=g, device="cuda").to(BF), s)
    return s


@pytest.mark.parametrize("rows,outs,cols", [(1, 8, 8), (40, 61, 40), (450, 64, 40), (3000, 24, 130), (700, 4096, 1100), (400, 4099, 1100)])
def test_weight_grad_of_one_row_for_all(zf, rows, outs, cols):
    """dy of row distance 0."""
    g = gen(outs)
    s, row = kept_input(zf, rows, cols, g), torch.randn(outs, generator=g, device="cuda").to(BF)
    a, b = torch.full((outs, cols), 7.0, device="cuda"), torch.empty(outs, cols, device="cuda")
    zf.zero_weight_grad8(row.expand(rows, outs), s, a)
    zf.zero_weight_grad8(row.expand(rows, outs).contiguous(), s, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("outs,cols", [(64, 40), (61, 40), (2048, 2048), (4096, 4096), (4099, 4001)])
@pytest.mark.parametrize("ld", [(1 << 25) - 8, 1 << 25, (1 << 25) + 1, (1 << 25) + 8])
def test_weight_grad_of_rows_far_apart(zf, outs, cols, ld):
    """Up to a distance of 2^25 the main loop's loads count bytes in 32 bits."""
    rows, g = 450, gen(cols)
    s, dy = kept_input(zf, rows, cols, g), torch.randn(rows, outs, generator=g, device="cuda").to(BF)
    far = torch.empty((rows - 1) * ld + outs, dtype=BF, device="cuda").as_strided((rows, outs), (ld, 1))
    far.copy_(dy)
    a, b = torch.full((outs, cols), 7.0, device="cuda"), torch.empty(outs, cols, device="cuda")
    zf.zero_weight_grad8(far, s, a)
    zf.zero_weight_grad8(dy, s, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("rows,outs,cols", [(20000, 33, 65), (30000, 130, 70), (65536, 64, 64)])
@pytest.mark.parametrize("dtype", (BF, H))
def test_weight_grad_over_many_rows_is_exact(zf, rows, outs, cols, dtype):
    """Codes of whole numbers and dy of -1, 0 and 1: sums are whole numbers below 65536 * 127 < 2^24."""
    g = gen(rows)
    s = zf.Saved8(rows, cols)
    s.codes.zero_()
    s.codes[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    s.exponents.fill_(133)
    dy = torch.randint(-1, 2, (rows, outs), generator=g, device="cuda").to(dtype)
    dy[:, 0], dy[:, 1] = 1, torch.where(s.codes[:, 0] < 0, -1, 1).to(dtype)          # and one that only grows
    grad = torch.empty(outs, cols, device="cuda")
    zf.zero_weight_grad8(dy, s, grad)
    want = torch.matmul(dy.double().t().contiguous(), s.codes[:, :cols].double())
    assert float(want[1, 0]) > 1e6 and torch.equal(grad.double(), want)
