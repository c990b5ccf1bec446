"""Which path a call of the attention over 4 bits takes, for tests to say that it is the one they mean."""
REQUESTS = 4096  # more are not cut into parts


def waves(D, R):
    """Waves of a part, for R query rows a head."""
    n = (R - 1) // (16 if R <= 16 or D == 256 else 32)
    return 1 if n == 0 else 2 if n == 1 else 4


def parts(D, R):
    """Parts that a sequence of pairs is cut into, without a shared part beside it."""
    return 256 * (3 if D == 64 else 2) * 4 // waves(D, R)


def taken(D, R, N, Hkv, own):
    """Whether few_kernel takes the requests' own keys, `own` tokens of each table."""
    return R <= 32 or (R <= 64 and N * Hkv * own >= {64: 3 << 18, 128: 7 << 15, 256: 7 << 14}[D])
