"""The linear layer's plan (kernel, tile width, K slices) and its items' rounds restated, for tests that
have to know which paths a size takes."""


def plan(M, N, K, b_mn, sms):
    """-> (pair, columns of a tile, slices, K blocks a slice) of the least estimated time"""
    num_kb = -(-K // 64)
    best = (float("inf"), None)

    def consider(pair, bn, tiles, workers, kb_us, fixed):
        nonlocal best
        for s in range(1, 17):
            if s > 1 and num_kb // s < 4:
                break
            per = -(-num_kb // s)
            if -(-num_kb // per) != s:
                continue
            join = 2.5 + 2.0 * s * M * N * 4 / 4e6 if s > 1 else 0
            us = fixed + float(-(-tiles * s // workers)) * per * kb_us + join
            if us < best[0]:
                best = (us, (pair, bn, s, per))

    if M > 128 and N > 64:
        for bn in range(256, 127, -32):
            loaded = -(-bn // 128) * 128 if b_mn else bn
            consider(True, bn, -(-M // 256) * -(-N // bn), sms // 2, max(0.27 * bn / 256, (16.0 + loaded / 16.0) / 100), 3)
    for bn in (128, 64):
        consider(False, bn, -(-M // 128) * -(-N // bn), sms, max(0.12, (16.0 * min(M, 128) / 128 + bn / 8.0) / 100), 4)
    return best[1]


def items(M, N, p):
    """Tiles times slices of a plan."""
    rows = 256 if p[0] else 128
    return -(-M // rows) * -(-N // p[1]) * p[2]


def work_item(k, c, C, n0, n1, rest, gap):
    """Item k of pair c of C of a launch of two products of n0 and n1 items: (product, item) or None."""
    n = (n0 - 1 - c) // C + 1 if c < n0 else 0
    if k < n:
        return 0, c + k * C
    k -= n
    if gap and c >= rest:
        if k < gap:
            i = k * (C - rest) + c - rest
            return (1, i) if i < n1 else None
        k -= gap
    i = gap * (C - rest) + k * C + c
    return (1, i) if i < n1 else None


def two_products(B, IC, OC, sms):
    """The backward pass's launch: (plans of dx and dW, items first and second, pairs, rest, gap), the first of
    the longer K; None where the two do not share a launch."""
    dx, dw = plan(B, IC, OC, True, sms), plan(OC, IC, B, True, sms)
    if not (dx[0] and dw[0]):
        return None
    n = [(items(B, IC, dx), dx), (items(OC, IC, dw), dw)]
    if dx[3] < dw[3]:
        n.reverse()
    pairs = min(sms // 2, n[0][0] + n[1][0])
    rest = n[0][0] % pairs
    gap = n[0][1][3] // n[1][1][3] if rest else 0
    return (dx, dw), n[0][0], n[1][0], pairs, rest, gap
