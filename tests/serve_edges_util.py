"""How chunk attention's tensor-core kernel walks its line of work, from the lengths."""


def waves_of(ctx, new, Hk, G, D, sms):
    """Waves that the kernel walks: where the row tiles of a head read its keys more than four
    times, as many as keep a wave's K and V below 64 MB and its part of the line of work at 64 key
    tiles a stretch or more."""
    pair, stretches = 2 * (128 // G), sms // 2 if D == 256 else sms
    line = walked = 0
    for c, n in zip(ctx, new):
        for t in range(0, n, pair):
            keys = c + min(t + pair, n)
            if n - t <= pair // 2:
                keys -= (keys + 4) // 5 - 1
            line, walked = line + (keys + 256) * Hk, walked + keys
    keys = sum(c + n for c, n in zip(ctx, new) if n)
    if walked <= 4 * keys:
        return 1
    return max(1, min(8, -(-keys * Hk * 4 * D // (64 << 20)), line // (stretches * 64 * 128)))
