"""Host replay of how the many-row kernel of paged attention cuts its work: items in order
on one line, equal runs of it, and the key tiles of each item's parts (no arithmetic of the
method)."""

CTAS, ROWS, TILE, ITEM_COST, MIN_TILES, SLOTS = 152, 256, 64, 12, 4, 4


def item_tiles(length, n, G, left=-1, right=-1):
    """Key tiles of the items of one row and KV head (0: its queries see no key)."""
    first = length - n

    def lo(i):
        return 0 if left < 0 else min(max(first + i - left, 0), length)

    def end(i):
        return length if right < 0 else min(max(first + i + right + 1, 0), length)

    tiles = []
    for r0 in range(0, n * G, ROWS):
        a, e = lo(r0 // G), end((min(r0 + ROWS, n * G) - 1) // G)
        tiles.append(-(-e // TILE) - a // TILE if e > a else 0)
    return tiles


def runs(lens, n, G, Hkv, left=-1, right=-1):
    """For each CTA the key tiles of its items' parts, in order."""
    items = [t for b in range(len(lens)) for _ in range(Hkv)
             for t in item_tiles(int(lens[b]), int(n[b]), G, left, right)]
    units = [ITEM_COST + max(t, 1) for t in items]
    per = max(-(-sum(units) // CTAS), MIN_TILES + ITEM_COST)
    parts = [[] for _ in range(CTAS)]
    at = 0
    for t, u in zip(items, units):
        for cta in range(at // per, (at + u - 1) // per + 1):
            x0, x1 = max(cta * per - at, 0), min((cta + 1) * per - at, u)
            if x1 > ITEM_COST:
                parts[cta].append(min(x1 - ITEM_COST, t) - max(x0 - ITEM_COST, 0))
        at += u
    return parts


def waits_for_itself(parts, with_empty_items):
    """Whether a loader, holding a tile that it has not delivered, looks for the tile two
    ahead (or the end) in a slot that the held tile's segment keeps from coming round."""
    segments = [t for t in parts if with_empty_items or t > 0]
    of_tile = [s for s, t in enumerate(segments) for _ in range(max(t, 0))]
    of_tile += [len(segments)] * 2
    return any(of_tile[i + 2] >= of_tile[i] + SLOTS for i in range(len(of_tile) - 2))
