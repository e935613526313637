"""Cases of the products with 4-bit weights that between them take every kind of
tile: with few rows, 32, 64, 128 and 160 to 256 rows. test_w4_choice.py checks on
the host that they do."""

# Over all tokens: N, and the numbers of tokens with the tiles that each takes
WIDE_N = {False: 16392, True: 8200}              # gated: half as many columns
TOKENS = {3: "few", 12: "few", 61: "32", 117: "64", 203: "128", 299: "160", 380: "192",
          437: "224", 509: "256"}
H = 288

# By expert: (counts, room for rows, columns not gated, gated)
_TALL = [(i * 37) % 256 + 1 for i in range(264)]
_CUT = [129 + i % 128 for i in range(100)]
_LOW = [32, 17, 1, 16, 25, 0, 31, 18, 20, 9] * 6
_FEW_LOW = [20, 1, 0, 3, 16, 2, 1, 1] * 5
_SOME = [240, 3, 256, 0, 16, 200, 1, 9, 150, 2]
EXPERTS = {
    # name: counts, rows, N, N gated, kernel, tiles
    "tall": (_TALL, 256, 248, 120, "big", {"32", "64", "128", "160", "192", "224", "256"}),
    "cut": (_CUT, 257, 248, 120, "big", {"128"}),
    "low": (_LOW, 32, 2056, 1032, "low", {"32"}),
    "low_and_few": (_FEW_LOW, 32, 2056, 1032, "low", {"few"}),
    "some": (_SOME, 261, 8200, 4104, "big", {"few", "160", "224", "256"}),
}
