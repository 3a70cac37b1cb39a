"""Which kernel form the 4-bit layer calls take for a problem: the library's
choice of tiles and splits (csrc/q4_tile.hpp tile_choose and the tables beside
its callers, csrc/q4.hip few_rows, csrc/q4_moe.hip moe_enqueue), written out
again so that a test can say which form it is meant to reach."""
import math

PROMPT = [(256, 256, 128.0), (128, 256, 80.0), (128, 128, 42.0), (64, 128, 28.0)]
GRAD = [(256, 256, 130.0), (128, 256, 88.0), (64, 256, 64.0)]


def ceil_div(a, b):
    return -(-a // b)


def tile_choose(shapes, T, cols, depth, most):
    """(tokens, columns) of the tile and the workgroups that share its terms."""
    best, least = None, 0.0
    for tokens, width, cost in shapes:
        tiles = ceil_div(T, tokens) * ceil_div(cols, width)
        s = 1
        while s == 1 or (s <= most and tiles * s <= 1024):
            us = (ceil_div(tiles * s, 256) * cost * depth / (4096.0 * s) +
                  (2.0 + 8.0e-6 / 4 * s * T * cols if s > 1 else 0.0))
            if least == 0.0 or us < least:
                least, best = us, (tokens, width, s)
            s += 1
    return best


def prompt_form(T, m, n):
    """q4_linear beyond 64 tokens."""
    return tile_choose(PROMPT, T, m, n, min(8, ceil_div(n, 128) // 2))


def grad_form(T, m, n):
    """q4_linear_grad."""
    return tile_choose(GRAD, T, n, m, min(16, ceil_div(m, 64) // 2))


def few_form(T, m):
    """q4_linear up to 64 tokens: quads of tokens and row tiles of a workgroup."""
    return next(q for q in (1, 2, 4, 8, 16) if T <= 4 * q), 2 if ceil_div(m, 16) >= 512 else 1


def moe_up_form(T, f, E, k):
    """q4_moe: waves per row tile of the up products."""
    waves = ceil_div(f, 16) * min(E, T * k)
    return 8 if 8 * waves <= 8192 else 4 if 4 * waves <= 8192 else 2


def moe_splits(T, h, f, E, k):
    """q4_moe: workgroups that share a row tile of the down products."""
    return max(1, min(4, ceil_div(256, ceil_div(h, 16)), min(E, T * k) * ceil_div(f, 128) // 32))
