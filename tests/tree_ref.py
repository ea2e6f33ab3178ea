"""Plain implementations of the tree calls, one node after the other, and trees to try them on."""


def ancestors(parent):
    """Each node's ancestors and itself, as a whole number's bits."""
    seen = []
    for i, p in enumerate(parent):
        seen.append((seen[p] if 0 <= p < i else 0) | 1 << i)
    return seen


def tree(rng, n, kind):
    """Parents of n nodes; "wild" has values that name no node ahead."""
    out = []
    for i in range(n):
        if kind == "chain":
            out.append(i - 1)
        elif kind == "star":
            out.append(0 if i else -1)
        elif kind == "roots":
            out.append(-1 if i == 0 or rng.random() < 0.3 else int(rng.integers(0, i)))
        elif kind == "wild":
            out.append(int(rng.integers(-3, i + 3)) if rng.random() < 0.7 else [-2 ** 31, 2 ** 31 - 1, i, 70000][int(rng.integers(0, 4))])
        else:
            out.append(int(rng.integers(max(0, i - 5), i)) if i else -1)
    return out


def plan(parents, ctx, T, N, gap=0):
    """POS and MASK (whole numbers) of T rows; parents: a list for each request; gap: rows ahead of the first."""
    pos, mask = [-1] * gap, [0] * gap
    for parent, c in zip(parents, ctx):
        anc = ancestors(parent[:N])
        pos += [min(max(c, 0) + bin(a).count("1") - 1, 2 ** 31 - 1) for a in anc] + [-1] * (len(parent) - len(anc))
        mask += anc + [0] * (len(parent) - len(anc))
    pad = max(0, T - len(pos))
    return (pos + [-1] * pad)[:T], (mask + [0] * pad)[:T]


def accept(parents, token, choice, written, N, first):
    """ACC, PATH and NEXT; token, choice and written by row, request r's rows from first[r]; rows behind them are none."""
    acc, path, after = [], [], []
    for parent, c0 in zip(parents, first):
        n = max(0, min(len(parent), N, len(token) - c0))
        at, took = 0 if n and written[c0] else -1, []
        while at >= 0:
            took.append(at)
            want = choice[c0 + at]
            at = next((j for j in range(at + 1, n) if parent[j] == at and written[c0 + j] and token[c0 + j] == want and want >= 0), -1)
        acc.append(len(took))
        path.append(took + [-1] * (N - len(took)))
        after.append(choice[c0 + took[-1]] if took else -1)
    return acc, path, after
