"""The 8-bit products' choice of a kernel, as the library's dispatch makes it, and
cases that between them run every kernel it can choose.

A kernel is (streaming | gemm, gate/up pair or one matrix, its tile, how the rows
come: coded by itself (1 or up to 4 rows), one matrix' rows, routed rows)."""


def _up(v, m):
    return -(-v // m)


def one_pass(T, k, E, routed, N, K, pair, codes=False):
    """The kernel of one pass: N channels (gate/up pairs if pair) over K inputs."""
    rows = T * k
    slots = min(E, rows) if routed else 1
    mean = _up(rows, slots)
    groups = _up(N, 16) * (2 if pair else 1)
    how = "routed" if routed else "rows"
    if not codes and not routed and T <= 4 and T * _up(K, 64) * 64 <= 24576:
        how = "coded 1" if T == 1 else "coded 4"
    else:
        ng = 2 if pair or slots * groups >= 256 else 1
        wgs = _up(groups, ng) * _up(mean, 16)
        if mean > 12 if slots > 1 else mean > 16 and wgs > 256:
            def fits(bm, cw):
                return ((bm == 32 or mean > bm // (4 if routed else 2))
                        and slots * _up(mean, bm) * _up(groups, 4 * cw) >= 160)
            for bm, cw, kp in ((128, 4, 1), (64, 4, 1), (64, 2, 2), (32, 4, 1), (32, 2, 2)):
                if fits(bm, cw):
                    return "gemm", pair, (bm, cw, kp), how
            return "gemm", pair, (32, 1, 4), how
    many = slots * groups
    if many >= 1024:
        tile = (2, 1, 8)
    elif many >= 256:
        tile = (2, 4, 8)
    else:
        tile = (2 if pair else 1, 8, 4)
    return "streaming", pair, tile, how


def ffn(T, k, E, routed, H, I):
    """The two kernels of a feed-forward on float rows (routed rows are coded by a
    launch of their own)."""
    return [one_pass(T, k, E, routed, I, H, True), one_pass(T, k, E, routed, H, I, False)]


# (T, K, N)
LINEAR = [
    (1, 72, 100), (3, 72, 100), (9, 72, 100),
    (1, 100, 4100), (1, 320, 6144), (3, 100, 4112), (9, 72, 4104),
    (1, 72, 16390), (3, 72, 16400), (9, 72, 16400),
    (337, 72, 179), (1305, 72, 387), (1273, 72, 770), (1412, 72, 792), (1418, 136, 1557),
    (300, 72, 13695),
]
# (T, H, I)
SHARED = [
    (1, 72, 40), (3, 72, 40), (9, 72, 40),
    (1, 72, 2056), (3, 72, 2048), (9, 72, 2056), (1, 72, 8200), (3, 72, 8192), (9, 72, 8200),
    (1, 4104, 72), (3, 4096, 72), (9, 4104, 72), (1, 16392, 40), (3, 16400, 40), (9, 16392, 40),
    (584, 146, 100), (1340, 390, 201), (1331, 780, 393), (1439, 810, 513), (1424, 1898, 795),
    (949, 4880, 40), (129, 72, 10223),
]
# (T, E, k, H, I)
ROUTED = [
    (4, 2, 1, 40, 41), (18, 65, 8, 72, 72), (8, 64, 8, 272, 272), (8, 64, 8, 264, 280),
    (51, 2, 1, 72, 44), (810, 5, 3, 146, 80), (1037, 12, 5, 72, 41), (990, 5, 5, 137, 70),
    (779, 81, 7, 72, 41), (320, 64, 8, 520, 272),
]
# (T, E, k, H, I, which experts the tokens take)
EXPERTS = [
    (5, 256, 8, 72, 40, "any"), (40, 256, 8, 40, 72, "blocks"), (500, 256, 8, 40, 40, "any"),
    (500, 256, 8, 40, 40, "blocks"),
    (7, 300, 8, 72, 40, "any"), (60, 300, 4, 40, 72, "far"), (64, 300, 2, 40, 40, "one"),
    (260, 300, 16, 40, 40, "any"), (260, 300, 16, 40, 40, "far"), (2000, 300, 2, 40, 40, "one"),
    (30, 1024, 8, 40, 40, "any"), (100, 1024, 16, 40, 40, "blocks"), (50, 1024, 2, 40, 40, "one"),
    (850, 1024, 16, 40, 40, "any"), (850, 1024, 16, 40, 40, "blocks"),
    (850, 1024, 16, 40, 40, "far"), (7000, 1024, 2, 40, 40, "one"),
]


def taken(E, which):
    """The experts that tokens choose from: all; some blocks of 64 only, the others
    empty, and the last expert; those past the first 256 (or 192); two."""
    if which == "any":
        return list(range(E))
    if which == "blocks":
        return [e for e in range(E) if e // 64 % 3 == 1] + [E - 1]
    if which == "far":
        return list(range(256 if E > 280 else 192, E))
    return [E // 3, E - 1]
