"""Which kernels the gradients of the 16-bit products take, by the rules of csrc/gemm_16_grad.hip, written again here so that
tests can say which of them their cases reach; tests/test_layer_plan_host.py holds them against the library's workspaces."""


def up(a, b):
    return -(-a // b)


def best_cut(narrow, wide, steps, one, memory, outputs, wide_parts, unaligned):
    """(256 x 256 tiles, parts) of the least estimate in us."""
    best, least = (False, 1), float("inf")
    for w in range(1 if unaligned else 2):
        for n in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32):
            if n > 1 and (2 * n > steps or (w and not wide_parts)):
                break
            each = up(steps, n)
            parts = 1 if n == 1 else up(steps, each)
            tiles = (wide if w else narrow) * parts
            step = 1.8 * up(tiles, 256) if w else (1.05 if unaligned else one) if tiles <= 256 else \
                (1.6 if unaligned else 1.1) * up(tiles, 512)
            us = max(step * each, memory) + (4 + 2e-6 * parts * outputs if parts > 1 else 0)
            if us < least:
                best, least = (bool(w), parts), us
    return best


def odd(M, N):
    return bool(M % 8 or N % 8)


def row_plan(S, E, M, N):
    """dA: (rows of a thin tile or 0, 256 x 256 tiles, parts); M rows of B a sum, N columns."""
    groups = max(min(E, S), 1)
    rows = S // groups
    high = 0 if groups > 1 or M * N > 1 << 23 else 16 if rows <= 16 else 32 if rows <= 32 else 0
    steps = up(M, 64)

    def tiles(bm, bn):
        return max((S // bm + groups if groups > 1 else up(S, bm)) * up(N, bn), 1)

    if high and tiles(high, 64) <= 1 << 21:
        want = min(512 // tiles(high, 64), steps // 4, 32)
        return high, False, 1 if want < 2 else up(steps, up(steps, want))
    even = [tiles(b, b) - (groups // 2 * up(N, b) if groups > 1 else 0) for b in (128, 256)]
    return (0, *best_cut(*even, steps, 0.55, 2.0 * groups * M * N / 5.5e6, S * N, False, odd(M, N)))


def grad_cut(S, E, M, N):
    """dB, M x N a matrix: (256 x 256 tiles, parts)."""
    tiles = [up(M, b) * up(N, b) * E for b in (128, 256)]
    return best_cut(*tiles, up(S // E, 64), 0.65, 0.0, E * M * N, True, odd(M, N))


def work_bytes(S, E, N, K, gated):
    M = 2 * N if gated else N
    dA, dB = row_plan(S, E, M, K)[2], grad_cut(S, E, M, K)[1]
    parts = max(dA * S * K if dA > 1 else 0, dB * E * M * K if dB > 1 else 0) * 4
    return parts + (S * up(2 * N, 64) * 64 * 2 if gated else 0)


def kernels(S, E, M, N, experts, gather, aligned):
    """The kernels of dA and of dB, as names."""
    high, wide, parts = row_plan(S, E, M, N)
    groups = min(E, S) if experts else 1
    tiles = (S // 128 + groups if experts else up(S, 128)) * up(N, 128)
    if high:
        a = "thin %d" % high
    elif not aligned or (parts == 1 and 2 * M < 16):
        a = "staged"
    elif wide:
        a = "256"
    else:
        a = "128, four steps" if (tiles * parts <= 256 or (parts == 1 and S <= 128 * groups)) else "128, two steps"
    b_wide, b_parts = grad_cut(S, E, M, N)
    b = "staged" if not aligned else "256" if b_wide else "128"
    return ("dA %s%s" % (a, " in parts" if parts > 1 else ""),
            "dB %s%s%s" % (b, " in parts" if b_parts > 1 else "", " of sources" if gather else ""))
