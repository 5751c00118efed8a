"""The size rules of the 8-bit projections, written again from their description: which
form a call takes.  Helpers of the tests that have to reach every form."""


def decode_form(M, K, sizes):
    """(16-token blocks, 16-column blocks) of a unit for up to 64 tokens: 32 columns where
    there are units enough."""
    units = sum(sizes) // 32
    few = 128 if K <= 2048 else 192 if K < 8192 else 448
    wide = units >= (few if M <= 16 else 256)
    return "decode", 1 if M <= 16 else 2 if M <= 32 else 4, 2 if wide else 1


def form(M, K, sizes, L):
    """("decode", tokens / 16, columns / 16), ("groups", columns / 16), ("units", rows,
    columns) or ("tiles",), with a table of L slots."""
    if M <= 64:
        return decode_form(M, K, sizes)
    N, groups = sum(sizes), -(-M // 64)
    if groups * -(-N // 32) <= 256 and K >= 2048:
        return "groups", 2 if groups * (N // 32) >= 192 else 1

    def rounds(rows, width):
        return -(-(-(-M // rows) * sum(-(-n // width) for n in sizes)) // 256)

    def met(rows):                       # segments that so many rows belong to
        return min(L, M, min(L, M) * rows // M + 1)
    small, large = rounds(64, 128) * (14 * 4096 + 85 * K), rounds(128, 256) * (80 * 4096 + 200 * K)
    tiles = rounds(256, 256) * (115 * 4096 + 330 * K + 10240 * met(256))
    if tiles < (small if small < large else large + rounds(128, 256) * 6144 * met(128)):
        return ("tiles",)
    return ("units", 64, 128) if small < large else ("units", 128, 256)


EVERY_FORM = {("decode", t, c) for t in (1, 2, 4) for c in (1, 2)} | {
    ("groups", 1), ("groups", 2), ("units", 64, 128), ("units", 128, 256), ("tiles",)}
