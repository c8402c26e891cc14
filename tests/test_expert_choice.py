"""Which kernel each product takes: the library's rule (expert.cpp, built for the CPU) over the
sizes that the GPU tests compare with the definitions, so that every kernel is among them."""
import os
import subprocess

import pytest

import expert_kernels as K
import expert_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bf16_fp8_weight_amd", "csrc")
SOURCES = [os.path.join(ROOT, "tests", "c_abi", "expert_choice.cpp"), os.path.join(ROOT, "tests", "sanitize", "plan_error_stub.cpp"),
           *(os.path.join(CSRC, f) for f in ("expert.cpp", "plan.cpp", "schedule.cpp", "host_api.cpp"))]
PLAIN, GATED, GATED_BACK = range(3)


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("choice") / "expert_choice")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-Wall", "-I", os.path.join(ROOT, "include"), "-I", CSRC, *SOURCES, "-o", exe,
                    "-lpthread"], check=True)

    def run(lines):
        r = subprocess.run([exe], input="\n".join(" ".join(str(x) for x in l) for l in lines) + "\n", capture_output=True,
                           text=True, timeout=60)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.split()

    return run


def _product(form, epi, lay, m, n, k, gathered=False, pad_a=2, pad_b=8):
    """As the GPU tests lay it out: without offsets for one expert, `pad` elements behind each row."""
    a, b = (m, n) if form == R.TN else (k, k if form == R.NT else n)
    return ("p", form, epi, lay.n_rows, len(lay.counts), int(len(lay.counts) > 1), 300 if gathered else -1, m, n, k, a + pad_a, b + pad_b)


def _mx(gated, lay, n, k):
    nb = -(-k // 32)
    return ("m", int(gated), lay.n_rows, len(lay.counts), int(len(lay.counts) > 1), n, k, 16 * nb + 16, (nb + 3) // 4 * 4 + 4,
            16 * nb + 16, (nb + 3) // 4 * 4 + 4)


ALIGNED = {"64split", "64x128", "128", "128wide", "256"}


@pytest.mark.parametrize("form", [R.NT, R.NN])
@pytest.mark.parametrize("gathered", [False, True])
def test_products(choose, form, gathered):
    got = choose([_product(form, PLAIN, lay, 0, n, k, gathered) for _, lay, n, k in K.PRODUCTS])
    assert got == [c[0] for c in K.PRODUCTS]
    assert set(got) == ALIGNED | {"any64", "any128", "16split"}


@pytest.mark.parametrize("gathered", [False, True])
def test_gradients_of_weights(choose, gathered):
    got = choose([_product(R.TN, PLAIN, lay, m, n, 0, gathered, 8, 2) for _, lay, m, n in K.GRADIENTS])
    assert got == [c[0] for c in K.GRADIENTS]
    assert set(got) == ALIGNED | {"any64", "any128"}


def test_gated(choose):
    forward = choose([_product(R.NT, GATED, lay, 0, n, k, pad_a=8, pad_b=2) for _, _, lay, n, k in K.GATED])
    back = choose([_product(R.NN, GATED_BACK, lay, 0, n, k) for _, _, lay, n, k in K.GATED])
    assert forward == [c[0] for c in K.GATED] and back == [c[1] for c in K.GATED]
    assert set(forward) == set(back) == ALIGNED | {"any64", "any128", "16split"}


def test_mxfp4(choose):
    for gated in (False, True):
        got = choose([_mx(gated, lay, n // 2 if gated else n, k) for _, lay, n, k in K.MXFP4])
        assert got == [c[0] for c in K.MXFP4]
        assert set(got) == {"32split", "64split", "128", "256"}  # any128: test_mxfp4_rows_far_apart
        assert choose([("m", int(gated), 33, 1, 0, 24, 70, 2 ** 22 + 16, 4, 2 ** 22 + 16, 4)]) == ["any128"]


def test_mxfp4_weights_beyond_31_bits(choose):
    """A plain product's tiles reach 256 rows, however long the matrix is; gated ones from the gate rows to the up rows."""
    rows, k = 2 ** 18 + 8, 2 ** 14  # 2 GiB of codes
    line = lambda gated, n, b_stride, scale: ("m", gated, 200, 1, 0, n, k, k // 2, k // 32, b_stride, scale)
    assert choose([line(0, rows, k // 2, k // 32), line(0, rows, k // 2, 2 ** 14), line(1, rows // 2 + 8, k // 2, k // 32)]) == ["128"] * 3
    assert choose([line(1, rows, k // 2, k // 32), line(1, rows, k // 2, 2 ** 14), line(0, 40, 2 ** 22 + 16, k // 32),
                   line(0, 40, k // 2, 2 ** 22 + 4)]) == ["any128"] * 4
    assert choose([line(0, 40, 2 ** 22, k // 32), line(0, 40, k // 2, 2 ** 22)]) != ["any128"] * 2


def test_the_largest_strides_and_sizes(choose):
    """No sum or product of the rule passes 64 bits (-ftrapv ends the program), and far rows take the kernels that reach them."""
    far = 2 ** 58
    for gated in (0, 1):
        base = ["m", gated, 2, 1, 0, 2 - gated, 70, 48, 4, 48, 4]
        lines = []
        for at in (7, 8, 9, 10):
            lines.append(base[:at] + [far] + base[at + 1:])
        assert choose(lines) == ["any128"] * 4
    big = 2 ** 24
    assert choose([("m", 0, 2 ** 20, 1024, 1, big, big, big // 2, big // 32, big // 2, big // 32)]) == ["any128"]
    assert choose([("p", R.TN, PLAIN, 2 ** 27, 1024, 1, -1, 2 ** 12, 2 ** 12, 0, 2 ** 12, 2 ** 12)]) == ["256"]
    assert choose([("p", R.TN, PLAIN, 2, 1, 0, -1, big, big, 0, far, far)]) == ["any128"]
    assert choose([("p", R.NT, PLAIN, 2 ** 20, 1024, 1, -1, 0, 2 ** 20, 64, 64, 64)]) == ["256"]
    assert choose([("p", R.NT, PLAIN, 2, 1, 0, 5, 0, 2, 64, 2 ** 56, far)]) == ["any64"]
