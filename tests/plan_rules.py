"""What the tests expect of the library's choices (csrc/plan.h), so that a test
of one variant says so.  test_host_plan.py holds these against the library's."""


def tile_rows(T: int, k: int, E: int, I: int, f32: bool) -> int:
    """Rows of a product tile of the experts: 32 (by 64 weight rows), 128 (float32) or 256 (bf16)."""
    pairs, large = T * k, 128 if f32 else 256
    tiles = max(pairs // large, E) * -(-2 * I // large)
    return 32 if pairs // E < 28 or tiles < 128 else large
