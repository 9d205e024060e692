"""The largest numbers of tiles of the bf16 and fp8 products (CPU only; pointers
are never dereferenced): device counts may claim the whole buffer for every
expert, and the table of tiles, with a workgroup's step behind the last one,
has to fit 32 bits."""
import pytest

import combine_dispatch_layout_amd as cdl
from test_products_abi import BF16, DX, EBIG, FAKE, FP8, GRAD, SWIGLU8

MOST = (1 << 31) - 1 - 256                    # rows, and tiles
# form, base arguments, output columns of a tile, the argument that is its width, by its kind
FORMS = [("cdl_grouped_bf16", BF16, 256, "N"), ("cdl_grouped_swiglu_bf16", BF16, 128, "N"),
         ("cdl_grouped_swiglu_bf16_grad", GRAD, 128, "N"), ("cdl_grouped_bf16_dx", DX, 256, "K"),
         ("cdl_grouped_fp8", FP8, 256, "N"), ("cdl_grouped_swiglu_fp8", SWIGLU8, 128, "N")]


def call(name, base, **over):
    args = dict(base)
    assert not set(over) - set(args)
    args.update(over)
    return getattr(cdl.library(), name)(*args.values())


@pytest.mark.parametrize("name,base,columns,width", FORMS)
def test_segments_that_may_all_claim_the_buffer(name, base, columns, width):
    """Row counts within their own limit, and more tiles than numbers whatever rows (128 to 256) a tile has."""
    tiles_n = (1 << 20) // columns
    assert 2048 * (MOST // 256) * tiles_n > MOST
    assert call(name, base, rows=MOST, L=2048, **{width: 1 << 20}) == EBIG
    # one row tile of the largest size too many (2^30 / 256 rows, 2048 experts: one column tile is too many)
    rows = 1 << 30
    assert rows // 256 * 2048 > MOST
    assert call(name, base, rows=rows, L=2048, **{width: columns}) == EBIG
    # the largest tile, to the row: L * row tiles * column tiles = 2^31 - 2
    L, m, n = 1302, 49981, 33
    assert L * m * n == (1 << 31) - 2
    assert call(name, base, rows=m * 256, L=L, **{width: n * columns}) == EBIG


@pytest.mark.parametrize("name,base,columns,width", FORMS)
def test_padded_buffers_of_too_many_tiles(name, base, columns, width):
    """L * cap rows: here every tile is one that a full buffer has."""
    L, n = 2048, (1 << 20) // columns
    cap = MOST // L
    assert L * (cap // 256) * n > MOST
    assert call(name, base, rows=L * cap, L=L, seg=None, cap=cap, **{width: 1 << 20}) == EBIG
    assert FAKE.value == 0x10000
