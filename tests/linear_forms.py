"""Sizes of the 4-bit product that take each form of its kernel, with several tiles per CTA.

(T, N, K) by form. The rule that picks the form gives small sizes to single tiles, so the sizes
here are chosen against it and both test suites check that the library takes the form named."""

ROWS, SINGLE, PAIR, WIDE = 0, 1, 2, 3
NAMES = {ROWS: "rows", SINGLE: "single", PAIR: "pair", WIDE: "wide"}

SIZES = {
    # 3 or 4 tiles per CTA; one and eight rows; one and several stages of 256 columns
    ROWS: [(3, 57000, 256), (8, 40008, 1024), (1, 38408, 2080)],
    # 387 and 440 tiles on 148 CTAs, whole and ragged stages
    SINGLE: [(316, 16400, 768), (2444, 2792, 256)],
    # 209, 219 and 240 tiles on 74 pairs: T mod 256 below 128 (the second CTA of the last tiles has no rows) and
    # above, N past whole tiles by 8 columns, one, three and nine stages; then 66 tiles of a long sum
    PAIR: [(2600, 4616, 544), (700, 18440, 544), (2368, 6144, 64), (2000, 5000, 2080), (1500, 2600, 12288)],
    # 144, 375 and 385 tiles on 148 CTAs, N mod 256 below and above 128, one to five stages
    WIDE: [(333, 12288, 800), (563, 19008, 1152), (850, 13968, 128)],
}
