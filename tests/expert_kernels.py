"""Sizes of the experts' products and, to each, the kernel that takes it. test_expert_choice
holds the library's rule to these names on the CPU; test_gpu_expert_kernels compares the
results with the definitions in 64 bits."""
import expert_ref as R

EIGHT = R.Layout([900, 0, 300, 257, 128, 1, 700, 515], align=16, lead=3, tail=5)
SIX = R.Layout([100, 0, 77, 200, 65, 64], lead=2, tail=40)
ODD = R.Layout([65, 0, 500, 64, 1, 129])
FEW = R.Layout([9, 0, 5])

# kernel, rows, columns of out, length of the sum: NT and NN alike
PRODUCTS = [
    ("any64", R.Layout([301, 0, 77]), 131, 77),
    ("any128", R.Layout([2101]), 2103, 133),
    ("16split", FEW, 1030, 3070),
    ("64split", R.Layout([500]), 1030, 1022),
    ("64split", SIX, 514, 286),
    ("64x128", R.Layout([701]), 2002, 202),
    ("64x128", R.Layout([300, 0, 257, 65, 64, 1], lead=1, tail=70), 1102, 998),
    ("128wide", R.Layout([1000]), 2050, 200),
    ("128wide", R.Layout([513, 0, 130, 257], lead=2, tail=9), 2050, 1030),
    ("128", R.Layout([1030]), 5640, 96),
    ("128", R.Layout([70] * 30 + [0, 129], align=128), 1100, 330),
    ("256", R.Layout([4100]), 4104, 134),
    ("256", EIGHT, 4002, 330),
]
# kernel, rows (the sum), rows and columns of out
GRADIENTS = [
    ("any64", R.Layout([77, 0, 300]), 131, 77),
    ("any128", R.Layout([77]), 2101, 2049),
    ("any128", ODD, 2101, 777),
    ("any64", R.Layout([10, 0, 12] * 21), 41, 49),
    ("any64", R.Layout([5, 0, 3] * 100), 65, 65),
    ("64split", R.Layout([10, 0, 12] * 21), 40, 48),
    ("64split", R.Layout([3000]), 130, 200),
    ("64split", SIX, 194, 130),
    ("64x128", R.Layout([300]), 702, 2000),
    ("64x128", R.Layout([31]), 1024, 2048),
    ("64x128", R.Layout([5, 0, 3] * 100), 64, 64),
    ("64x128", R.Layout([70, 9] * 20), 200, 200),
    ("128wide", R.Layout([300]), 1030, 2052),
    ("128wide", R.Layout([513, 0, 130, 257], lead=2, tail=9), 642, 1030),
    ("128", R.Layout([333]), 2050, 2052),
    ("128", R.Layout([300, 0, 500, 33, 7]), 1026, 1030),
    ("128", R.Layout([70, 100] * 12), 640, 640),
    ("256", R.Layout([70]), 4100, 4106),
    ("256", EIGHT, 1026, 2052),
]
# kernel of the forward pass, of the backward pass, rows, columns of h, length of the sum
GATED = [
    ("any64", "any64", R.Layout([301, 0, 77]), 130, 77),
    ("any128", "any128", R.Layout([2101]), 2102, 133),
    ("16split", "16split", FEW, 514, 3070),
    ("64split", "64split", R.Layout([500]), 514, 1022),
    ("64x128", "64split", SIX, 1026, 286),
    ("128wide", "64x128", R.Layout([701]), 2002, 202),
    ("128wide", "64x128", R.Layout([300, 0, 257, 65, 64, 1], lead=1, tail=70), 1102, 998),
    ("128", "128wide", R.Layout([1000]), 2050, 200),
    ("256", "128", R.Layout([1030]), 5640, 96),
    ("128", "128", R.Layout([70] * 30 + [0, 129], align=128), 1100, 330),
    ("256", "256", R.Layout([4100]), 4104, 134),
    ("256", "256", EIGHT, 4002, 330),
]
# kernel, rows, columns, length of the sum: as sums, and gated with half as many columns of h
MXFP4 = [
    ("32split", R.Layout([60]), 1032, 3000),
    ("32split", FEW, 1032, 1111),
    ("64split", R.Layout([500]), 2000, 1000),
    ("64split", SIX, 1032, 3000),
    ("128", R.Layout([1030]), 2600, 200),
    ("128", R.Layout([70] * 30 + [0, 129], align=128), 1100, 1300),
    ("128", R.Layout([4100]), 4104, 1000),
    ("128", EIGHT, 4000, 3583),
    ("256", R.Layout([4100]), 4104, 3584),
    ("256", EIGHT, 4000, 3633),
]


def name(case):
    return "-".join([c for c in case if isinstance(c, str)] + ["x".join(str(c) for c in case if isinstance(c, int))])
