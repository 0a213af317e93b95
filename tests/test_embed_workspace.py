"""The embedding gradient's workspace on both sides of what it depends on (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    return m


@pytest.mark.parametrize("n,dim", [(0, 0), (0, 4096), (1, 1), (2048, 1), (2048, 512), (1024, 2048), (512, 8192), (1, 1 << 24)])
def test_few_tokens_need_none(zf, n, dim):
    for vocab in (0, 1, 70000, 1 << 25):
        assert zf.zero_embed_grad_workspace(n, vocab, dim) == 0


# a tile is 128 sorted positions from n * ceil(dim / 512) = 65536 on, and 32 before; each has two fp32 rows
@pytest.mark.parametrize("n,dim,tile", [(2049, 1, 32), (2049, 512, 32), (2048, 513, 32), (1025, 2048, 32), (65535, 512, 32), (65536, 512, 128),
                                        (32767, 1024, 32), (32768, 513, 128), (8191, 4096, 32), (8192, 4096, 128),
                                        (100000, 1000, 128)])
def test_bytes(zf, n, dim, tile):
    for vocab in (1, 50021):
        rows = 2 * -(-n // tile) * (-(-dim // 8) * 8) * 4
        counts = (-(-n // 1024) + 1) * 1024
        least = 16 * n + vocab + rows + counts
        assert least <= zf.zero_embed_grad_workspace(n, vocab, dim) <= least + 8 * 256
        # as documented: 17 bytes a token and 2 KiB, one a row, an fp32 row per 16 tokens or per 64, and two
        assert zf.zero_embed_grad_workspace(n, vocab, dim) <= 17 * n + 4096 + vocab + (n / (tile / 2) + 2) * (dim + 7) * 4
