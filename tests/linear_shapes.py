"""Shapes (tokens, inputs, outputs) by the kernel that the 4-bit linear map runs
for them: odd counts, outputs that end inside a block, one and several chunks of
inputs, one and several token passes."""
SHAPES = {
    "tile 16x16 w8": [(3, 16512, 64), (31, 1152, 64), (127, 1024, 48)],
    "tile 16x32 w4": [(3, 1024, 4128), (130, 384, 2064)],
    "tile 16x32 w8": [(2, 1152, 4112)],
    "tile 16x48 w8": [(300, 1152, 528), (5, 1152, 8208)],
    "tile 32x32 w4": [(2501, 1408, 64)],
    "tile 32x48 w4": [(63, 2560, 4112)],
    "tile 32x64 w4": [(387, 640, 976)],
    "tile 32x96 w4": [(70, 2176, 12304)],
    "tile 48x64 w4": [(515, 2048, 4112), (33, 640, 13696)],
    "tile 64x64 w4": [(191, 4224, 4112)],
    # one chunk; several, with more row tiles than the totals of 256 blocks hold
    "stream 16": [(3, 3200, 26608), (13, 6272, 196624)],
    "stream 32 short": [(17, 1664, 50480), (63, 1920, 49344)],
    "stream 32": [(19, 5248, 25712), (70, 4096, 50304), (63, 8192, 50304)],
    "gemm 64": [(1500, 640, 4112)],
    "gemm 96": [(2501, 640, 2064), (2501, 4096, 4112)],
    "gemm 128": [(1500, 256, 8208), (3001, 2048, 4112)],
}
LISTED = [(name, *s) for name, shapes in SHAPES.items() for s in shapes]
# one shape a kernel, a small one
EACH = [(name, *shapes[0]) for name, shapes in SHAPES.items()]
