"""GDR_VALIDATE when one of its own runtime calls is refused: the call fails,
rather than taking the input for valid.  The runtime's calls are replaced by
fakes in a process of its own (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import pytest

import gated_delta_rule_37_gb300 as gdr
from gated_delta_rule_37_gb300 import build as gbuild

FAKE = r"""
#include <stddef.h>
#include <stdlib.h>
#include <string.h>
static unsigned word;
static int last;
static int answer(const char* name) {
    const char* fails = getenv("FAILS");
    return last = fails && !strcmp(fails, name) ? 999 : 0;
}
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int which, int d) { *v = which == 75 ? 10 : which == 76 ? 3 : 152; return 0; }
int cudaGetSymbolAddress(void** p, const void* symbol) { *p = &word; return 0; }
int cudaMemsetAsync(void* p, int v, size_t n, void* s) { return answer("memset"); }
int __cudaLaunchKernel() { static int calls; return calls++ ? 0 : answer("launch"); }
int cudaGetLastError(void) { int e = last; last = 0; return e; }
int cudaMemcpyAsync(void* d, const void* s, size_t n, int kind, void* stream) { return answer("copy"); }
int cudaStreamSynchronize(void* s) { return answer("wait"); }
const char* cudaGetErrorString(int e) { return "refused"; }
"""

CALL = r"""
import ctypes, sys
P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
lib = ctypes.CDLL(sys.argv[1])
lib.gdr_last_error.restype = ctypes.c_char_p
lib.gdr_linrec_step.argtypes = [P, I64, P, I64, P, I, I, P, P, I, I64, I, I, I, I, P, I64, P, I, P]
code = lib.gdr_linrec_step(256, 64, 512, 64, 768, 1, 8, 1024, 1280, 4, 4, 64, 0, 1, int(sys.argv[2]), 1536, 64, None, 0, None)
print(code, lib.gdr_last_error().decode())
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    gbuild.build()
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.c").write_text(FAKE)
    subprocess.run([cc, "-std=gnu11", "-shared", "-fPIC", "-w", "-o", str(d / "fake.so"), str(d / "fake.c")], check=True)
    return str(d / "fake.so")


def step(fake, flags, fails=""):
    env = dict(os.environ, LD_PRELOAD=fake, FAILS=fails)
    r = subprocess.run([sys.executable, "-c", CALL, gdr.LIB_PATH, str(flags)], env=env, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, r.stderr
    code, _, message = r.stdout.strip().partition(" ")
    return int(code), message


def test_the_fakes_answer(fake):
    """A call of accepted input goes through, with and without validation."""
    assert step(fake, gdr.GDR_COMMIT) == (0, "")
    assert step(fake, gdr.GDR_COMMIT | gdr.GDR_VALIDATE) == (0, "")


@pytest.mark.parametrize("fails", ["memset", "launch", "copy", "wait"])
def test_a_refused_call_is_not_a_valid_input(fake, fails):
    code, message = step(fake, gdr.GDR_COMMIT | gdr.GDR_VALIDATE, fails)
    assert code == 4 and message.startswith("validation"), (code, message)
