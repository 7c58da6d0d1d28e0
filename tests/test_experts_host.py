"""The host side of the products' launches against a stand-in for the CUDA
runtime (fake_cudart.c), without a GPU: the library's own objects, linked with
it, on several devices and with calls of the runtime that fail."""
import ctypes
import glob
import os
import subprocess

import pytest
import torch

import combine_ep_plan_gb300 as ep
from combine_ep_plan_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 1 << 20  # device pointers: nothing reads them
PAIR, NARROW, THIN = "matmul_pair", "matmul_narrow", "matmul_thin"


class Launch(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("grid", ctypes.c_uint), ("block", ctypes.c_uint), ("cluster", ctypes.c_uint),
                ("smem", ctypes.c_size_t), ("overlaps", ctypes.c_int), ("name", ctypes.c_char * 256)]


def link(out, objects):
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-fPIC", "-c", os.path.join(HERE, "fake_cudart.c"),
                    "-I", cuda, "-o", out + ".o"], check=True)
    # -Bsymbolic: torch has brought the real runtime into the process
    subprocess.run(["g++", "-shared", "-Wl,-z,defs", "-Wl,-Bsymbolic", "-o", out, out + ".o", *objects, "-lpthread"], check=True)
    lib = ctypes.CDLL(out)
    lib.fake_status.restype = ctypes.POINTER(ctypes.c_uint)
    lib.fake_launch.restype = ctypes.POINTER(Launch)
    lib.fake_fail.argtypes = [ctypes.c_char_p, ctypes.c_int, ctypes.c_int]
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.ep_matmul_int8.argtypes = [vp, vp, i64, vp, vp, i32, i64, i64, vp, vp, i32, vp, i64, vp]
    lib.ep_matmul_status.argtypes = [vp]
    return lib


def built_objects():
    build.build()
    names = [os.path.join(build.BUILD, os.path.basename(s) + ".o") for s in build.sources()]
    if not all(os.path.exists(n) for n in names):
        build.build(force=True)
    assert sorted(names) == sorted(n for n in glob.glob(os.path.join(build.BUILD, "*.o")) if n in names)
    return names


@pytest.fixture()
def lib(tmp_path):
    """A copy of its own for each test: what the library keeps starts anew."""
    lib = link(str(tmp_path / "libep_fake.so"), built_objects())
    lib.fake_reset()
    return lib


# rows of a product 512 -> 4096 with 8 experts, by the kernel that takes it
ROWS = {PAIR: 4000, NARROW: 500, THIN: 40}


def product(lib, rows, dtype=ep.EP_DTYPE_BF16, E=8):
    return lib.ep_matmul_int8(FAKE, FAKE, rows, FAKE, FAKE, E, 4096, 512, FAKE, None, dtype, FAKE, rows, None)


def launches(lib):
    return [lib.fake_launch(i).contents for i in range(lib.fake_launches())]


@pytest.mark.parametrize("dtype", [ep.EP_DTYPE_BF16, ep.EP_DTYPE_F32])
@pytest.mark.parametrize("kernel", [PAIR, NARROW, THIN])
def test_every_device_launches_every_product_kernel(lib, kernel, dtype):
    """A kernel's limit of shared memory belongs to the device it was raised on."""
    for device in (0, 1, 0, 3):
        lib.fake_use_device(device)
        assert product(lib, ROWS[kernel], dtype) == ep.EP_OK
    got = launches(lib)
    assert [g.device for g in got] == [0, 1, 0, 3] and all(kernel in g.name.decode() for g in got)
    assert all(g.smem > 48 * 1024 for g in got) or kernel == THIN


def test_pairs_fill_the_device_that_runs_them(lib):
    """The number of pairs that run at once is asked of each device, and does not
    depend on the first call's experts."""
    for device, experts in ((0, 2048), (1, 8), (0, 8)):
        lib.fake_use_device(device)
        assert product(lib, 500000, E=experts) == ep.EP_OK
    assert [g.grid for g in launches(lib)] == [120, 122, 120]


@pytest.mark.parametrize("kernel", [PAIR, NARROW])
@pytest.mark.parametrize("call", ["cudaFuncSetAttribute", "cudaGetDriverEntryPointByVersion", "cudaGetDevice",
                                  "cudaOccupancyMaxActiveClusters"])
def test_a_failure_is_not_kept(lib, kernel, call):
    lib.fake_fail(call.encode(), 999, 1)
    if call == "cudaOccupancyMaxActiveClusters" and kernel == NARROW:
        pytest.skip("not called by this kernel")
    first = product(lib, ROWS[kernel])
    assert first == ep.EP_ERR_CUDA or call in ("cudaGetDevice", "cudaOccupancyMaxActiveClusters")  # a default serves
    assert product(lib, ROWS[kernel]) == ep.EP_OK
    last = launches(lib)[-1]
    assert kernel in last.name.decode()
    if kernel == PAIR:
        assert product(lib, 500000) == ep.EP_OK and launches(lib)[-1].grid == 120


def test_a_launch_that_is_refused_is_reported(lib):
    lib.fake_fail(b"cudaLaunchKernelExC", 2, 1)
    assert product(lib, ROWS[PAIR]) == ep.EP_ERR_OOM
    assert product(lib, ROWS[PAIR]) == ep.EP_OK


@pytest.mark.parametrize("kernel", [PAIR, NARROW, THIN])
@pytest.mark.parametrize("ahead", [True, False])
def test_launches_overlap_only_where_kernels_wait(tmp_path, kernel, ahead):
    """Built with EP_USE_PDL=0 no kernel waits for the one ahead of it, so none
    may start before that has ended."""
    objects = built_objects()
    if not ahead:
        name = next(o for o in objects if "ep_matmul_kernels" in o)
        plain = str(tmp_path / "plain.o")
        ptx_only = ["-gencode", "arch=compute_103a,code=compute_103a"]  # nothing runs: no machine code
        subprocess.run([build.nvcc(), *ptx_only, *build.NVCC_FLAGS, "-DEP_USE_PDL=0", "-c",
                        os.path.join(build.CSRC, "ep_matmul_kernels.cu"), "-o", plain], check=True)
        objects[objects.index(name)] = plain
    lib = link(str(tmp_path / "libep_fake.so"), objects)
    lib.fake_reset()
    for rows in (ROWS[kernel], 5):
        assert product(lib, rows) == ep.EP_OK
    got = launches(lib)
    assert kernel in got[0].name.decode() and [g.overlaps for g in got] == [int(ahead)] * 2
    assert got[0].cluster == (2 if kernel == PAIR else 1)


TIMEOUT, CAPACITY = 8, 4  # bits of the status word


def test_a_status_that_comes_in_while_another_is_read_is_kept(lib):
    """A product on another stream may record an error between the read and the clearing."""
    for first, late, codes in ((CAPACITY, TIMEOUT, (ep.EP_ERR_CAPACITY, ep.EP_ERR_TIMEOUT)),
                               (TIMEOUT, CAPACITY, (ep.EP_ERR_TIMEOUT, ep.EP_ERR_CAPACITY))):
        lib.fake_status()[0] = first
        lib.fake_late(late)
        assert tuple(lib.ep_matmul_status(None) for _ in codes) == codes
        assert lib.ep_matmul_status(None) == ep.EP_OK


def test_two_errors_are_two_reports(lib):
    lib.fake_status()[0] = TIMEOUT | CAPACITY
    assert [lib.ep_matmul_status(None) for _ in range(3)] == [ep.EP_ERR_TIMEOUT, ep.EP_ERR_CAPACITY, ep.EP_OK]


def test_each_device_has_its_status(lib):
    lib.fake_status()[0] = CAPACITY
    lib.fake_use_device(1)
    assert lib.ep_matmul_status(None) == ep.EP_OK
    lib.fake_use_device(0)
    assert lib.ep_matmul_status(None) == ep.EP_ERR_CAPACITY and lib.ep_matmul_status(None) == ep.EP_OK


@pytest.mark.parametrize("call", ["cudaLaunchKernelExC", "cudaGetSymbolAddress", "cudaStreamSynchronize", "cudaMemcpyAsync"])
def test_a_status_that_cannot_be_read_is_an_error(lib, call):
    lib.fake_status()[0] = CAPACITY
    lib.fake_fail(call.encode(), 999, 1)
    assert lib.ep_matmul_status(None) == ep.EP_ERR_CUDA


@pytest.mark.parametrize("out,error", [([[0.0]], TypeError), ("bf16", TypeError), (torch.zeros(()), ValueError),
                                       (torch.zeros(4, 8, dtype=torch.float16), TypeError)])
def test_an_output_of_the_wrong_kind_is_refused_as_such(out, error):
    class Handle:
        T, K, E, A = 4, 1, 2, 1
    with pytest.raises(error, match="out must be"):
        ep.expert_matmul_int8(Handle(), torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4),
                              torch.zeros(2, 8, 16, dtype=torch.int8), torch.zeros(2, 8), out=out)
