"""Sizes [M, N] of mx_linear's tests by the kernel that takes them (csrc/linear_plan.h;
test_linear_plan.py checks that they are still there)."""

KERNELS = ["direct", "split 32x32", "split 32x64", "split 64x32", "split 64x64", "tile 128", "tile 256"]

# aligned rows of the output in both types, except where a width is odd
SHAPES = {
    "direct": [(1, 7168), (4, 96), (16, 4096), (13, 264)],
    "split 32x32": [(32, 7168), (64, 2048), (20, 5000), (256, 1000)],
    "split 32x64": [(32, 10000), (25, 8300)],
    "split 64x32": [(128, 4096), (48, 6000), (500, 1000)],
    "split 64x64": [(256, 4096), (45, 9000), (500, 2056)],
    "tile 128": [(1100, 2304), (1091, 2312), (1100, 2300)],
    "tile 256": [(2048, 8192), (2040, 8184), (2040, 8190)],
}
