"""Calls of lb_norm by the shape that they are launched in: the GPU tests make them, a CPU test holds that they are such
calls.  Threads of a row x pieces of 8 columns of each -> (rows, width)."""

SHAPES = {
    (64, 1): [(5, 40), (2050, 511)],
    (64, 3): [(2049, 1031), (2048, 520), (2500, 1536), (2051, 513)],
    (256, 1): [(2047, 1031), (7, 2041)],
    (512, 1): [(300, 4096), (257, 2049)],
    (512, 2): [(300, 8192), (257, 4099), (256, 8185)],
    (1024, 1): [(255, 4099), (255, 8192)],
    (1024, 2): [(260, 8193), (3, 16384)],
    (1024, 4): [(2, 16385), (64, 30001)],
}
CALLS = [(shape, *call) for shape, calls in SHAPES.items() for call in calls]
