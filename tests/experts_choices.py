"""Sizes that take each of the experts' kernels, first and second: (tokens, experts, experts a token,
inputs) by the weights' types (0 bfloat16, 1 e4m3 with row scales, 2 with block scales, 3 8-bit
integers). No width is a whole number of 128 bytes' stages. Where there is one expert and more than one
choice, tokens name it twice. The two last widths of the first list are those beyond which tiles of 4
rows stream x."""

CHOICES = {
    (0, 1, 2, 3): ((1, 24, 8, 272), (1, 24, 8, 12816), (5, 6, 3, 272), (5, 6, 3, 4112), (5, 6, 3, 6416),
        (5, 6, 3, 7568), (9, 2, 2, 1936), (9, 2, 2, 3216), (9, 2, 2, 3696), (21, 67, 2, 9040), (29, 1, 1, 272),
        (37, 16, 2, 3216), (37, 16, 2, 5264), (37, 16, 2, 6416), (64, 1, 2, 1424), (64, 1, 2, 1712),
        (70, 300, 2, 272), (100, 32, 1, 272), (3, 64, 4, 14416), (70, 300, 2, 14416)),
    (1, 2, 3): ((29, 1, 1, 2832), (33, 9, 3, 2832), (33, 9, 3, 3216), (40, 2, 2, 1712), (64, 1, 2, 272),
        (70, 1, 1, 784), (70, 300, 2, 6416), (70, 300, 2, 10512), (100, 6, 2, 272)),
    (0,): ((9, 2, 2, 272), (29, 1, 1, 1040), (29, 1, 1, 1424), (29, 1, 1, 1712), (33, 9, 3, 272), (64, 1, 2, 784),
        (70, 1, 1, 272), (70, 300, 2, 7024), (70, 300, 2, 11792), (120, 13, 1, 1712), (120, 13, 1, 2832),
        (120, 13, 1, 3216)),
}
