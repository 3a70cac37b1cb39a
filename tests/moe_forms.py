"""Which kernel form the experts' products take for a problem: the library's
choice (csrc/q4_experts.hip experts_plan, experts_grad_plan, experts_run),
written out again so that a test can say which form it is meant to reach."""
from q4_forms import ceil_div

FEW_MEAN = 48
PRODUCT = [(256, 256, (128.0, 80.0, 56.0)), (128, 128, (39.0, 28.0, 28.0)), (64, 128, (28.0, 28.0, 28.0))]
GRAD = [(256, 256, (130.0, 88.0, 64.0)), (128, 128, (44.0, 32.0, 32.0))]


def choose(shapes, R, E, cols, depth, deepest):
    """(rows, columns) of the largest tile, the workgroups that share its depth ("tail":
    only those of the last tiles), and the time that is expected of it."""
    some, best = min(R, E), None
    for rows, width, us in shapes:
        work = tile = 0.0
        for q in range(8):
            c = max(1, int((0.475 + 0.15 * q) * R / some))
            rest = c % rows
            cut = 0.0 if rest == 0 else us[2 if rest <= rows // 4 else 1 if rest <= rows // 2 else 0]
            work += c // rows * us[0] + cut
            tile = max(tile, us[0] if c >= rows else cut)
        work *= some * ceil_div(cols, width) / (8.0 * 256)
        s = 1
        while s == 1 or (s <= deepest and (R // rows + some) * ceil_div(cols, width) * s <= 2048):
            t = max(work + 0.4 * tile / s, tile / s) * depth / 4096 + (2.0 + 8.0e-6 / 4 * s * R * cols if s > 1 else 0.0)
            if best is None or t < best[3]:
                best = rows, width, s, t
            s += 1
        if rows == 256:
            us256, whole, few = us[0] * depth / 4096, work, work <= 3.5 * tile
    t = whole * depth / 4096 + 0.1 * us256 + 20.0
    return (256, 256, "tail", t) if us256 >= 40.0 and few and t < best[3] else best


def tail(counts, cols, us, deepest):
    """Of a product whose tail is shared out, experts' rows given: whole tiles, the tiles
    of the tail, the parts of each, and which bodies (256, 128, 64 rows) they have."""
    rest = [c % 256 for c in counts]
    bodies = [256] * sum(c // 256 + (c % 256 > 128) for c in counts) + [128] * sum(64 < c <= 128 for c in rest) + \
        [64] * sum(0 < c <= 64 for c in rest)
    nc = ceil_div(cols, 256)
    tiles, us = len(bodies) * nc, int(100 * us)
    left, parts, best = tiles % 256, 1, us
    for s in range(2, deepest + 1):
        t = ceil_div(left * s, 256) * us // s + 200 + 9 * left * s
        if left * s <= 512 and t < best:
            best, parts = t, s
    return tiles - left, left, parts, {bodies[i // nc] for i in range(tiles - left, tiles)}


def experts_form(R, E, m, n):
    """q4_experts: ("few", waves of a pair of row tiles) or (rows, splits, sums): with
    sums beside the products where x's rows are aligned."""
    if R <= FEW_MEAN * E:
        waves = ceil_div(ceil_div(m, 16), 2) * min(R, E)
        return "few", 8 if 8 * waves <= 8192 else 4 if 4 * waves <= 8192 else 2
    rows, _, splits, us = choose(PRODUCT, R, E, m, n, min(8, ceil_div(n, 128) // 2))
    return rows, splits, rows == 64 and n % 64 == 0 and us < 30.0


def experts_grad_form(R, E, m, n, group):
    """q4_experts_grad: ("few" or a tile's rows, the workgroups that share a block's depth)."""
    best = choose(GRAD, R, E, n, m, min(16, ceil_div(m, 64) // 2))
    rows, some = 16 if group // 64 % 2 else 32, min(R, E)
    blocks = max(some, R // rows + some // 2)
    groups = blocks * ceil_div(n, 128)
    splits = max(1, min(16, 512 // groups, ceil_div(m, 32) // 16))
    if blocks * float(m) * n / ((4.2e6 if rows == 16 else 5.6e6) * min(1.0, groups * splits / 512.0)) <= 3.0 + best[3]:
        return "few", splits
    return best[0], best[2]
