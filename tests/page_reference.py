"""The pool's bookkeeping one sequence and one page after the other (plain Python)."""


def fork(page, width, src_seq, dst_seq, ref, table, held, length):
    status = []
    dsts = list(dst_seq)
    for i, (s, t) in enumerate(zip(src_seq, dst_seq)):
        ok = 0 <= s < len(held) and 0 <= t < len(held) and t not in dsts[:i] and s not in dsts
        if ok:
            used = -(-length[s] // page)
            ok = length[s] >= 0 and used <= min(held[s], width) and held[t] == 0
            ok = ok and all(0 <= p < len(ref) for p in table[s][:used])
        status.append(0 if ok else -1)
        if ok:
            table[t] = table[s][:used] + [-1] * (width - used)
            for p in table[s][:used]:
                ref[p] += 1
            held[t], length[t] = used, length[s]
    return status


def reserve(page, width, need, ref, table, held, length):
    """status and the copies (src, dst)."""
    S = len(held)
    want = [-(-(length[s] + need[s]) // page) for s in range(S)]
    fits, shared = [False] * S, [None] * S
    for s in range(S):
        fits[s] = need[s] > 0 and length[s] >= 0 and want[s] <= width and held[s] <= width and \
            length[s] <= held[s] * page
        if fits[s] and length[s] % page:
            p = table[s][length[s] // page]
            fits[s] = 0 <= p < len(ref)
            if fits[s] and ref[p] > 1:
                shared[s] = p
    askers = {}
    for s, p in enumerate(shared):
        if p is not None:
            askers.setdefault(p, []).append(s)
    copies = [p is not None and not (len(askers[p]) == ref[p] and askers[p][-1] == s) for s, p in enumerate(shared)]
    free = [p for p, r in enumerate(ref) if r <= 0]
    status, moves, asked = [], [], 0
    for s in range(S):
        demand = max(want[s] - held[s], 0) + copies[s] if fits[s] else 0
        asked += demand
        if need[s] <= 0:
            status.append(0)
        elif not fits[s]:
            status.append(-1)
        elif asked > len(free) and (demand or shared[s] is not None):
            status.append(-2)
        else:
            status.append(0)
            mine = free[asked - demand:asked]
            if copies[s]:
                old, new = table[s][length[s] // page], mine.pop(0)
                table[s][length[s] // page] = new
                ref[old] -= 1
                ref[new] = 1
                moves.append((old, new))
            for c, p in zip(range(held[s], want[s]), mine):
                table[s][c] = p
                ref[p] = 1
            held[s] = max(held[s], want[s])
    return status, moves


def free(drop, ref, table, held, length):
    for s, gone in enumerate(drop):
        if gone:
            for p in table[s][:held[s]]:
                if 0 <= p < len(ref):
                    ref[p] -= 1
            table[s] = [-1] * len(table[s])
            held[s] = length[s] = 0


def compact(most, ref, table):
    """moves and remap."""
    total = sum(r > 0 for r in ref)
    moves = list(zip([p for p in range(total, len(ref)) if ref[p] > 0], [p for p in range(total) if ref[p] <= 0]))[:most]
    remap = list(range(len(ref)))
    for s, t in moves:
        remap[s] = t
        ref[t], ref[s] = ref[s], 0
    for row in table:
        row[:] = [remap[p] if 0 <= p < len(ref) else p for p in row]
    return moves, remap
