"""The kernels' division by numbers that a call has once (Div in csrc/cross.h), on the CPU: against
the machine's, at every border of the quotient for small and large numbers."""
import os
import subprocess

from sparse_head_self_gb300 import _native
from sparse_head_self_gb300.build import CSRC

PROGRAM = r"""
#include "cross.h"
#include <cstdio>
#include <random>
using namespace fibatt;
int main() {
    const int64_t most = 2147483647;
    std::mt19937 r(1);
    long wrong = 0;
    const auto divisor = [&](int64_t d) {
        const Div by((uint32_t)d);
        const auto check = [&](int64_t n) {
            if (n >= 0 && n <= most) wrong += by.of((int)n) != n / d || by.rest((int)n) != n % d;
        };
        for (int64_t q : {int64_t(0), int64_t(1), int64_t(2), int64_t(3), int64_t(1000), most / d / 2, most / d - 1, most / d})
            for (int e = -2; e < 3; ++e) check(q * d + e);
        for (int i = 0; i < 50; ++i) check((int64_t)(r() >> 1)), check((int64_t)(r() >> 1 >> r() % 31));
        check(most);
    };
    for (int64_t d = 1; d < 20000; ++d) divisor(d);
    for (int s = 1; s < 31; ++s)
        for (int e = -3; e < 4; ++e)
            if ((1ll << s) + e > 0) divisor((1ll << s) + e);
    for (int i = 0; i < 20000; ++i) divisor(1 + (int64_t)(r() >> 1) % most);
    divisor(most);
    printf("%ld\n", wrong);
}
"""


def test_quotients_and_remainders(tmp_path):
    src, exe = tmp_path / "div.cpp", tmp_path / "div"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, "-I", os.path.dirname(_native.HEADER), "-I", cuda, "-o", str(exe),
                    str(src)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "0\n"
