"""Batches with more than twice as many tiles as the card has workgroups (256), for every kernel and direction of the grouped
products and every tile of the updates: a workgroup goes from tile to tile, of other experts and other numbers of rows."""
WORKGROUPS = 256
LONG, SHORT, FEW = [300, 0, 1, 257, 520] * 12, [161, 1, 40, 0, 90] * 24, [1, 0, 3, 8, 2] * 12
RAGGED = [0, 3, 33, 70, 1] * 12
# direction, rows of each expert, in, out, the kernel (variants.h: 0 any, 1 stream, 2 of 160 rows, 3 of 256)
PRODUCTS = [("y", LONG, 72, 1600, 3), ("y", SHORT, 72, 1600, 2), ("y", SHORT, 71, 1599, 0), ("y", FEW, 136, 448, 1),
            ("dx", LONG, 1600, 72, 3), ("dx", SHORT, 1600, 72, 2), ("dx", SHORT, 1599, 71, 0), ("dx", FEW, 448, 136, 1),
            ("int8", LONG, 200, 1600, 3), ("int8", SHORT, 200, 1599, 2), ("int8", FEW, 300, 448, 1)]
GRADIENTS = [(RAGGED, 520, 520), (RAGGED, 521, 517)]
# n, shorter side, longer side
UPDATES = [(300, 200, 300), (600, 100, 130), (300, 100, 130), (200, 33, 130), (600, 200, 200), (180, 352, 360), (600, 33, 64)]
