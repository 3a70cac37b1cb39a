"""Which kernel form the experts' products take for a problem: the library's
choice (csrc/q4_experts.hip experts_plan, experts_grad_plan, experts_run),
written out again so that a test can say which form it is meant to reach."""
from q4_forms import ceil_div

FEW_ROWS = 32
PRODUCT = [(256, 256, (128.0, 80.0, 56.0)), (128, 128, (42.0, 28.0, 28.0))]
GRAD = [(256, 256, (130.0, 88.0, 64.0))]


def estimate(shape, R, E, cols, depth, splits):
    rows, width, us = shape
    some = min(R, E)
    c, nc = R / some, ceil_div(cols, width)
    tile, one = us[0], c / rows * us[0] + 0.25 * (us[1] + us[2])
    if c <= rows // 4:
        tile = one = us[2]
    elif c <= rows // 2:
        tile = one = us[1]
    work = max(some * nc * one / 256 + 0.4 * tile / splits, tile / splits)
    return work * depth / 4096 + (2.0 + 8.0e-6 / 4 * splits * R * cols if splits > 1 else 0.0)


def choose(shapes, R, E, cols, depth, deepest):
    """(rows, columns) of the largest tile and the workgroups that share its depth."""
    best, least = None, 0.0
    for shape in shapes:
        s = 1
        while s == 1 or (s <= deepest and (R // shape[0] + min(R, E)) * ceil_div(cols, shape[1]) * s <= 2048):
            us = estimate(shape, R, E, cols, depth, s)
            if least == 0.0 or us < least:
                least, best = us, (shape[0], shape[1], s)
            s += 1
    return best


def experts_form(R, E, m, n):
    """q4_experts: ("few", waves of a pair of row tiles) or (rows, columns, splits)."""
    if R <= FEW_ROWS * E:
        waves = ceil_div(ceil_div(m, 16), 2) * min(R, E)
        return "few", 8 if 8 * waves <= 8192 else 4 if 4 * waves <= 8192 else 2
    return choose(PRODUCT, R, E, m, n, min(8, ceil_div(n, 128) // 2))


def experts_grad_form(R, E, m, n):
    """q4_experts_grad."""
    return choose(GRAD, R, E, n, m, min(16, ceil_div(m, 64) // 2))
