"""Page tables, slots and offsets of a step from request lengths, one request after the other in plain Python numbers."""
TOP = 2 ** 31 - 1


def plan(lens, new, table, page, stack, count, t, done=None):
    """Lists in; what ``kv_plan`` returns and leaves in the table and on the stack, as lists."""
    n, n_pages = len(lens), len(stack)
    table, stack = [list(r) for r in table], list(stack)
    width = len(table[0]) if n else 0
    cap = width * page
    have = [min(max(x, 0), cap) for x in lens]
    free = min(max(count, 0), n_pages)
    for s in range(n):
        if done is not None and done[s]:
            for p in table[s][:-(-have[s] // page)]:
                if 0 <= p < n_pages and free < n_pages:
                    stack[free] = p
                    free += 1
            have[s] = 0
    slots, positions, cu_q, cu_k, after = [], [], [0], [0], []
    lacking = 0
    for s in range(n):
        fresh = min(max(new[s], 0), t - len(slots))
        for pos in range(have[s], have[s] + fresh):
            slot = -1
            if pos < cap:
                if pos % page == 0:
                    p = -1
                    if free:
                        free -= 1
                        p = stack[free]
                    else:
                        lacking += 1
                    table[s][pos // page] = p if 0 <= p < n_pages else -1
                p = table[s][pos // page]
                if 0 <= p < n_pages:
                    slot = p * page + pos % page
            slots.append(slot)
            positions.append(pos)
        after.append(have[s] + fresh)
        cu_q.append(len(slots))
        cu_k.append(min(cu_k[-1] + after[-1], TOP))
    slots += [-1] * (t - len(slots))
    positions += [0] * (t - len(positions))
    return {"slots": slots, "positions": positions, "cu_q": cu_q, "cu_k": cu_k, "lens": after, "count": [free, lacking],
            "table": table, "stack": stack}
