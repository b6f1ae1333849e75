"""Inputs of mx_tree_attention that take each of its kernels, named by the rows
of its tiles: test_tree_plan_host.py holds them to the plan, test_gpu_tree_windows.py
runs them.  The choice goes by the rows and by the most keys that a row may see:
what the page table has room for, and under a window that many and `max_new`
(which is for speed only, any value is right), so a wide table and a large
`max_new` take small sequences to the kernels of large ones."""
from __future__ import annotations

# (nodes, keys) of each sequence, one KV head of four query heads
FEW = [(40, 500), (90, 91), (33, 260)]      # 217 rows on average
FEWER = [(20, 500), (31, 333), (25, 26)]    # 101

# rows per tile -> (sequences, keys that the table has room for, max_new)
WINDOWED = {16: (FEW, 0, None), 32: (FEW, 1 << 17, 40000), 128: (FEWER, 1 << 20, 1 << 22), 256: (FEW, 1 << 20, 1 << 22)}
WINDOWS = (1, 5, 64, 100, 450, 5000)

# contexts that are cut into parts, the first of them under a window as well
LONG = {16: ([(20, 9000), (15, 4000)], 0, None), 32: ([(60, 9000), (50, 4000)], 100000, 100000),
        128: ([(30, 9000), (28, 4000)], 1 << 20, 1 << 22), 256: ([(60, 9000), (50, 4000)], 1 << 20, 1 << 22)}
LONG_WINDOWS = (0, 2500, 3333)

# one sequence of so many parts that they are joined in two steps (16 and 32 rows), or by a kernel of their own
MANY = {16: ([(4, 17000)], 0, None), 32: ([(16, 30000)], 1 << 20, None), 128: ([(25, 17000)], 1 << 20, None), 256: ([(50, 17000)], 1 << 20, None)}


def width(case, page):
    """Columns of the table."""
    seqs, keys, _ = case
    return max(max(-(-L // page) for _, L in seqs) + 1, -(-keys // page))


def plans():
    """(rows per tile, sequences, page size, columns, window, max_new) of every call."""
    for cases, windows in ((WINDOWED, WINDOWS), (LONG, LONG_WINDOWS), (MANY, (0,)), (SHORT, (0, 5))):
        for rows, case in cases.items():
            for page in (2, 16):
                for window in windows:
                    most = max(n for n, _ in case[0]) if case[2] is None else case[2]
                    yield rows, case[0], page, width(case, page), window, most

# rows that see few keys, none or a few of a context
SHORT = {16: ([(40, 43), (90, 90), (33, 60)], 0, None), 32: ([(40, 43), (90, 90), (33, 60)], 40000, 40000),
         128: ([(20, 23), (31, 31), (25, 40)], 1 << 20, 1 << 22), 256: ([(40, 43), (90, 90), (33, 60)], 1 << 20, 1 << 22)}
