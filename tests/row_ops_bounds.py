"""Error bounds of the RMS norm counted from how its launches deal a row and a column.

U = 2^-24 is the rounding of one fp32 operation; a sum whose longest chain of additions has
k steps is off by at most k U times the sum of the terms' magnitudes."""
U = 2.0 ** -24


def serial(c: int) -> int:
    """Elements of a row that one thread adds one after the other: at most 48 up to 32,768
    channels (short rows lie with 2 to 16 threads of up to 32 elements, 8-bit rows up to 1536
    with a warp of 48), c / 1024 above."""
    return 48 if c <= 32768 else -(-c // 1024)


def rstd_bound(c: int) -> float:
    """Relative: the chain is a thread's own elements, 5 steps across a warp and at most 7
    across warps; the sum's rounding, the quotient and the addition of eps follow.  The root
    halves these.  rsqrtf is off by at most 2 last bits (4 U), the rounded x + residual by U."""
    return ((serial(c) + 5 + 7 + 3) / 2 + 4 + 1) * U


def norm_bound(c: int) -> float:
    """Relative, of the unrounded result: two products and the rounded x + residual besides."""
    return rstd_bound(c) + 3 * U


def dx_bound(c: int) -> float:
    """Of rstd (|g| + |xh| mean |g xh|) + |dsum|: the dot's chain (at most 16 elements a
    thread, c / 1024 above 16,377 channels, then 5 + 5 steps), xh, g, the products and
    the mean, and the final operations."""
    own = 16 if c <= 16377 else -(-c // 1024)
    return (own + 10 + 8) * U


def row_groups(c: int, item: int, per_thread: int) -> int:
    """Rows a CTA of the gradient has in work: 512 threads in groups of as many threads, a
    power of two, as hold a row's elements (whole items: a row that starts anywhere may touch
    one more)."""
    span = c if c % item == 0 else c + item - 1
    threads = 2
    while threads < 512 and threads * per_thread < span:
        threads *= 2
    return 512 // threads


def column_bound(n: int, c: int, item: int, per_thread: int) -> float:
    """Of the sum over rows of |dy xh|: a thread adds its rows of at least 144 CTAs (up to 4
    turns where one CTA takes all), then at most 4 steps across a warp, 15 across a CTA's
    groups, ceil(296 / 32) across the CTAs and 5 in the end; two roundings a product."""
    rows = row_groups(c, item, per_thread)
    return (max(4, -(-n // (144 * rows))) + 4 + 15 + 10 + 5 + 2) * U
