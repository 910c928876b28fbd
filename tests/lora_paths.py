"""Which kernels a forward call of ep_lora runs, as ep_lora.cu decides it, for
tests that are about one kind of them."""
from __future__ import annotations


def few_rows(pairs: int, E: int, rank: int) -> bool:
    """One kernel for few rows an adapter; else a shrink and an expand kernel."""
    if rank > 64 or pairs == 0:
        return False
    each = 256 if rank <= 16 else (64 if rank <= 32 else 16)
    return pairs <= max(each * E, 2048 if rank <= 32 else 128)


# What the function above restates; tests compare it with the source.
RULE = """\
    if (rank > kFewRank || rows.pairs == 0 || rows.num_rows == 0)
        return false;
    const int64_t each = rank <= 16 ? 256 : (rank <= 32 ? 64 : 16), all = rank <= 32 ? 2048 : 128;
    return rows.pairs <= std::max(each * rows.E, all);
"""
