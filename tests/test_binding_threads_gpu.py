"""The compiled binding lets other Python threads run while a call allocates and launches: a
full launch queue blocks a launch, and may itself wait for a host function that needs Python.
A copy of the module is given entry points that wait (5 s at most) until another Python thread
has been seen to run; no kernel is launched."""
import ctypes
import importlib.machinery
import importlib.util
import shutil
import subprocess
import threading
import time

import pytest
import torch

from paged_kv_cache_70_gb300 import build

pytestmark = pytest.mark.gpu

WAITS = """
#include <stddef.h>
#include <time.h>
static volatile int inside, released;
int entered(void) { return __atomic_load_n(&inside, __ATOMIC_SEQ_CST); }
void release(void) { __atomic_store_n(&released, 1, __ATOMIC_SEQ_CST); }
void reset(void) { inside = released = 0; }
int entry(void) {
    __atomic_store_n(&inside, 1, __ATOMIC_SEQ_CST);
    for (int i = 0; i < 5000; ++i) {
        if (__atomic_load_n(&released, __ATOMIC_SEQ_CST)) return 0;
        struct timespec t = {0, 1000000};
        nanosleep(&t, 0);
    }
    return -1;
}
size_t size(void) { return 256; }
"""


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    (d / "waits.c").write_text(WAITS)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(d / "waits.c"), "-o", str(d / "waits.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "waits.so"))
    build.build_binding()
    copy = str(d / "_pagedkv.so")  # (with entry points of its own)
    shutil.copy(build.binding_path(), copy)
    loader = importlib.machinery.ExtensionFileLoader("_pagedkv", copy)
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_pagedkv", loader))
    loader.exec_module(m)

    def check(func, status):
        raise RuntimeError(f"{func}: no other thread ran")

    at = lambda name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
    m.bind(check, at("entry"), at("entry"), at("entry"), at("entry"), at("size"))
    return lib, m


def calls(m):
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(3, 2, 64, device="cuda")
    cs = torch.zeros(9, 64, device="cuda")
    table, idx = torch.zeros(3, 2, **i32), torch.zeros(3, **i32)
    kc = torch.zeros(2, 4, 2, 64, device="cuda")
    k8 = torch.zeros(2, 2, 4, 64, device="cuda").to(torch.float8_e4m3fn)
    s = torch.zeros(2, 2, device="cuda")
    rest = (None, None, False, None)
    return {
        "write_rope": lambda: m.write(k, k, cs, table, idx, idx, kc, kc, None, None, k, *rest),
        "write_q8": lambda: m.write(k, k, None, table, idx, idx, k8, k8, s, s, None, *rest),
        "read_q8": lambda: m.read_q8(k8, k8, s, s, idx, torch.float32, None, None),
        "decode_q8": lambda: m.decode_q8(k, k8, k8, s, s, table, idx, None, None, None),
    }


@pytest.mark.parametrize("name", ["write_rope", "write_q8", "read_q8", "decode_q8"])
def test_another_thread_runs_meanwhile(waits, name):
    lib, m = waits
    call = calls(m)[name]
    lib.reset()

    done = threading.Event()

    def other():
        while not lib.entered() and not done.is_set():
            time.sleep(0.001)
        lib.release()

    t = threading.Thread(target=other)
    t.start()
    try:
        call()  # (raises if it waited in vain)
    finally:
        done.set()
        t.join(10)
