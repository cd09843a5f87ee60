"""Which bound of kv_precise a tree's attention has: that of V unpacked for many rows, or that of the
codes with p s in two parts (one or two tiles of 16 rows per wave)."""


def shares_unpacked_values(rows, dim, group):
    """rows: query rows per cached head."""
    return rows >= (256 if dim == 128 else 1024) and not (dim == 128 and group >= 64)
