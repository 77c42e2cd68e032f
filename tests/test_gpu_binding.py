"""The C++ part of the Python binding by itself: a copy of the module, whose C entries
are stand-ins."""

import ctypes
import importlib.machinery
import importlib.util
import shutil
import subprocess
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

# Entries that wait, two seconds at most, until another Python thread has had its turn.
STANDINS = r"""
#include <stddef.h>
#include <unistd.h>
volatile int turn = 0;
int entry(void) {
  for (int i = 0; i < 2000 && !turn; ++i) usleep(1000);
  return turn ? 0 : -5;
}
size_t workspace(void) { return 256; }
"""


@pytest.fixture(scope="module")
def standins(tmp_path_factory):
    """(module, library): the binding bound to the stand-ins."""
    from fp4_fp8_quant_gb300 import iq
    at = tmp_path_factory.mktemp("binding")
    (at / "entries.c").write_text(STANDINS)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(at / "entries.so"), str(at / "entries.c")], check=True)
    lib = ctypes.CDLL(str(at / "entries.so"))
    copy = str(at / "binding.so")
    shutil.copy(iq.BINDING_PATH, copy)
    loader = importlib.machinery.ExtensionFileLoader("_iq_torch", copy)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_iq_torch", loader=loader))
    address = lambda name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
    module.bind(*[address("workspace" if name.endswith("workspace") else "entry") for name in iq._ENTRIES])
    return module, lib


def calls():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    return {"quant_rows": (z(4, 128), z(3, t=i32), None, None, None),
            "route": (z(5, 8, t=f32), 2, 0, False, 1.0, None, None),
            "grouped_gemm": (z(4, 128, t=u8), z(1, 4, t=i32), z(2, 64, 128, t=u8), z(2, 1, 1, t=u8), z(3, t=i32), False, None, None, None),
            "combine": (z(4, 64), z(2, 2, t=i32), z(2, 2, t=f32), None, None, None),
            "adapters": (z(4, 64), None, z(1, 8, 64), z(1, 64, 8), z(1, t=f32), z(2, t=i32), z(1, t=i32), None, None, None)}


@pytest.mark.parametrize("name", ["quant_rows", "route", "grouped_gemm", "combine", "adapters"])
def test_other_threads_run_while_a_call_launches(cuda_device, standins, name):
    module, lib = standins
    turn = ctypes.c_int.in_dll(lib, "turn")
    turn.value = 0
    args = calls()[name]
    torch.cuda.synchronize()

    def take_turn():
        time.sleep(0.02)
        turn.value = 1

    other = threading.Thread(target=take_turn)
    other.start()
    result = getattr(module, name)(*args)
    other.join()
    assert not isinstance(result, int) and result is not None


def test_an_allocation_that_fails_raises_what_pytorch_raises(cuda_device):
    from fp4_fp8_quant_gb300 import iq
    x = torch.zeros((1, 1 << 16), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(1 << 24, dtype=torch.int32, device="cuda")       # 1.1 TB of codes
    with pytest.raises(torch.OutOfMemoryError):
        iq.fp8_quant_1x128_ue8m0(x, rows=rows)


def test_large_results_do_not_keep_one_another(cuda_device):
    """Past 1 MiB each result has memory of its own, up to there one allocation."""
    from fp4_fp8_quant_gb300 import iq
    x, l = torch.zeros((9, 7168), dtype=torch.bfloat16, device="cuda"), torch.zeros((9000, 16), device="cuda")
    size = lambda t: t.numel() * t.element_size()
    for M in (10, 2000):
        results = [iq.fp8_quant_1x128_ue8m0(x, rows=torch.zeros(M, dtype=torch.int32, device="cuda")), iq.moe_route(l[:M * 4 + 1000], 8)]
        for parts in results:
            held = [t.untyped_storage().nbytes() for t in parts]
            if M == 2000:
                assert held == [size(t) for t in parts] and len({t.untyped_storage().data_ptr() for t in parts}) == len(parts)
            else:
                assert max(held) <= 1 << 20 and len({t.untyped_storage().data_ptr() for t in parts}) == 1


def test_calls_of_several_threads_at_once(cuda_device):
    """Threads with a stream each, whose calls meet in the binding and the library:
    every result is that of the call by itself."""
    from fp4_fp8_quant_gb300 import iq
    gen = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda")
    w = torch.randint(0, 0x60, (4, 512, 2560), generator=gen, device="cuda", dtype=torch.uint8)
    w_sf = torch.full((4, 4, 20), 115, dtype=torch.uint8, device="cuda")
    a, b, scale = normal(2, 16, 2560).bfloat16(), normal(2, 256, 16).bfloat16(), torch.ones(2, device="cuda")
    bounds, used = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 7, 30], [1, 0]))
    inputs = [(normal(30, 2560).bfloat16(), normal(30, 4)) for _ in range(3)]

    def block(x, logits, stream=None):
        r = iq.moe_route(logits, 2, normalize=True, stream=stream)
        xq, xs = iq.fp8_quant_1x128_ue8m0(x, rows=r.rows, stream=stream)
        h = iq.grouped_gemm(xq, xs, w, w_sf, r.row_start, gated=True, stream=stream)
        y = iq.moe_combine(h, r.slots, r.weights, stream=stream)
        return iq.adapters(x, y, a, b, scale, bounds, used, stream=stream)

    want = [block(*i) for i in inputs]
    torch.cuda.synchronize()
    got = [[] for _ in inputs]

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(40):
            got[i].append(block(*inputs[i], stream=stream))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(inputs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(len(g) == 40 and all(torch.equal(o, v) for o in g) for g, v in zip(got, want))
    assert iq.device_status() == 0
