"""Rows of an output tile (128, 192 or 256) that the bf16 and fp8 products take
for a call's sizes, by the rule at product_tile_rows in products.hip: what a
test needs in order to reach each size."""

LDS = 160 * 1024


def _lds(fp8, rows):
    stages_a, stages_b = (2, 2) if rows == 256 else (3, 2) if rows == 192 else (3, 3)
    return stages_a * 256 * 128 + stages_b * rows * 128 + (3 * (rows * 16 + 256) + 2 * rows * 4 if fp8 else 0)


def tile_rows(rows, L, width, fp8=False, swiglu=False, quantised=False, padded=False):
    """width: output columns (SwiGLU: of the activations)."""
    fits = {m: _lds(fp8, m) + 4 * L <= LDS for m in (128, 192, 256)}
    if padded:
        return 192 if fits[192] else 256
    tiles_n = -(-width // (128 if swiglu else 256))
    r, best, least = rows / L, 256, None
    for m in (256, 192, 128):
        if not fits[m] or (m == 256 and quantised and fits[192]):
            continue
        tm = -(-rows // m) if L == 1 else 1.0 if r <= 0.8 * m else r / m + 0.5
        rounds = tm * L * tiles_n / 256
        cost = (1.0 if rounds <= 1 else 2.0 if rounds <= 2 else rounds) * {128: 1.03, 192: 1.33, 256: 1.59}[m]
        if least is None or cost < least:
            best, least = m, cost
    return best


def tiles(rows_of_experts, rows, width, swiglu=False):
    """Output tiles of a call."""
    return sum(-(-c // rows) for c in rows_of_experts) * -(-width // (128 if swiglu else 256))
