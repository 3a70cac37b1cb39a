"""Which kernel form the experts' products take for a problem: the library's
choice (csrc/q4_experts.hip experts_plan, experts_grad_plan, experts_run),
written out again so that a test can say which form it is meant to reach."""
from q4_forms import GRAD, PROMPT, ceil_div

FEW_ROWS = 32


def blocks_about(R, E, tokens):
    some = min(R, E)
    return max(some, R // tokens + some // 2)


def choose(shapes, R, E, cols, depth, most):
    """(rows, columns) of the tile and the workgroups that share its terms."""
    best, least = None, 0.0
    for tokens, width, cost in shapes:
        tiles = blocks_about(R, E, tokens) * ceil_div(cols, width)
        s = 1
        while s == 1 or (s <= most and tiles * s <= 1024):
            us = (ceil_div(tiles * s, 256) * cost * depth / (4096.0 * s) +
                  (2.0 + 8.0e-6 / 4 * s * R * cols if s > 1 else 0.0))
            if least == 0.0 or us < least:
                least, best = us, (tokens, width, s)
            s += 1
    return best


def experts_form(R, E, m, n):
    """q4_experts: ("few", waves of a pair of row tiles) or (rows, columns, splits)."""
    if R <= FEW_ROWS * E:
        waves = ceil_div(ceil_div(m, 16), 2) * min(R, E)
        return "few", 8 if 8 * waves <= 8192 else 4 if 4 * waves <= 8192 else 2
    return choose(PROMPT, R, E, m, n, min(8, ceil_div(n, 128) // 2))


def experts_grad_form(R, E, m, n):
    """q4_experts_grad."""
    return choose(GRAD, R, E, n, m, min(16, ceil_div(m, 64) // 2))
