"""Oracle for the paging of the caches (the definitions in include/rope_attention.h (g)).
Test infrastructure only (see the package docstring).  Python integers, request by request."""
from __future__ import annotations

import numpy as np


def _pages(n, block_size):
    return -(-n // block_size)


def extend(new_tokens, seq_lens, table, free_pages, free_count, *, block_num, block_size, max_tokens) -> dict:
    """index, cu_seqlens, new_seq_lens, table (a copy), new_free_count and errors."""
    table = np.array(table)
    cap = table.shape[1] * block_size
    avail = min(max(int(free_count), 0), block_num)
    index, cu, lens, errors, asked, rows, left = [], [0], [], 0, 0, 0, avail
    for b in range(len(seq_lens)):
        n, old = max(int(new_tokens[b]), 0), min(max(int(seq_lens[b]), 0), cap)
        rows += n
        ok = old + n <= cap and rows <= max_tokens
        if ok:
            want = _pages(old + n, block_size) - _pages(old, block_size)
            asked += want
            ok = want == 0 or asked <= avail
            if ok:
                for i in range(want):
                    left -= 1
                    table[b, _pages(old, block_size) + i] = free_pages[left]
        errors += not ok and n > 0
        lens.append(old + n if ok else old)
        for pos in range(old, old + min(n, max(0, max_tokens - len(index)))):
            slot = -1
            if ok:
                page = int(table[b, pos // block_size])
                if 0 <= page < block_num:
                    slot = page * block_size + pos % block_size
                else:
                    errors += 1
            index.append(slot)
        cu.append(min(rows, max_tokens))
    index += [-1] * (max_tokens - len(index))
    return {"index": np.array(index, np.int64), "cu_seqlens": np.array(cu, np.int32), "new_seq_lens": np.array(lens, np.int32),
            "table": table, "new_free_count": left, "errors": errors}


def slots(starts, counts, table, *, block_num, block_size, max_tokens) -> dict:
    """index, cu_seqlens and errors."""
    index, cu, rows, errors = [], [0], 0, 0
    for b in range(len(counts)):
        first, n = max(int(starts[b]), 0) if starts is not None else 0, max(int(counts[b]), 0)
        rows += n
        for pos in range(first, first + min(n, max(0, max_tokens - len(index)))):
            page = int(table[b, pos // block_size]) if pos < table.shape[1] * block_size else -1
            good = 0 <= page < block_num
            index.append(page * block_size + pos % block_size if good else -1)
            errors += not good
        cu.append(min(rows, max_tokens))
    index += [-1] * (max_tokens - len(index))
    return {"index": np.array(index, np.int64), "cu_seqlens": np.array(cu, np.int32), "errors": errors}


def truncate(keep, seq_lens, table, free_pages, free_count, *, block_num, block_size) -> dict:
    """new_seq_lens, free_pages (a copy), new_free_count and errors."""
    free = np.array(free_pages)
    cap = table.shape[1] * block_size
    count = min(max(int(free_count), 0), block_num)
    back, lens, errors = [], [], 0
    for b in range(len(seq_lens)):
        old = min(max(int(seq_lens[b]), 0), cap)
        new = 0 if keep is None else min(max(int(keep[b]), 0), old)
        lens.append(new)
        for page in table[b, _pages(new, block_size):_pages(old, block_size)].tolist():
            if 0 <= page < block_num:
                back.append(page)
            else:
                errors += 1
    room = min(len(back), block_num - count)
    errors += len(back) - room
    for i in range(room):
        free[count + room - 1 - i] = back[i]
    return {"new_seq_lens": np.array(lens, np.int32), "free_pages": free, "new_free_count": count + room, "errors": errors}
