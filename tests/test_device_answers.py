"""What a device is asked for once (csrc/clef_kernels.h, AskedOnce), compiled for the host with a CUDA runtime of the test's
own: answers are kept for their device and key, and a question that failed is asked again."""
import os
import re
import subprocess

from w8a8_quantized_projections_gb300 import build

CSRC = os.path.join(build.HERE, "csrc")
PROGRAM = r"""
#include "clef_kernels.h"
#include <cstdio>
int device = 0, asked = 0, cleared = 0;
cudaError_t device_status = cudaSuccess, status = cudaSuccess;
int clusters[70];
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return device_status; }
extern "C" cudaError_t cudaGetLastError() { ++cleared; return status; }
clef::AskedOnce<3> known;
int failures = 0;
#define EXPECT(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); ++failures; } } while (0)
cudaError_t get(int key, int *n) { return known.get(key, n, [&](int *m) { ++asked; *m = clusters[device] + key; return status; }); }
int main() {
    int n = 0;
    for (int d = 0; d < 70; ++d) clusters[d] = 100 + d;
    EXPECT(get(1, &n) == cudaSuccess && n == 101 && asked == 1);
    EXPECT(get(1, &n) == cudaSuccess && n == 101 && asked == 1);                       // kept
    EXPECT(get(2, &n) == cudaSuccess && n == 102 && asked == 2);                       // another key
    device = 3;
    EXPECT(get(1, &n) == cudaSuccess && n == 104 && asked == 3);                       // another device
    device = 0;
    EXPECT(get(1, &n) == cudaSuccess && n == 101 && asked == 3);
    device = 66;                                                                       // past the table: asked each time
    EXPECT(get(0, &n) == cudaSuccess && n == 166 && get(0, &n) == cudaSuccess && asked == 5);
    device = 5;                                                                        // a failure is not kept
    status = cudaErrorMemoryAllocation;
    EXPECT(get(0, &n) == cudaErrorMemoryAllocation && n == 0 && cleared == 1);
    status = cudaSuccess;
    EXPECT(get(0, &n) == cudaSuccess && n == 105);
    device = 6;                                                                        // nor is an answer of nothing
    clusters[6] = 0;
    EXPECT(get(0, &n) != cudaSuccess && n == 0 && cleared == 2);
    clusters[6] = 9;
    EXPECT(get(0, &n) == cudaSuccess && n == 9);
    device_status = cudaErrorNoDevice;
    EXPECT(get(0, &n) == cudaErrorNoDevice);
    return failures;
}
"""


def test_answers_belong_to_their_device(tmp_path):
    (tmp_path / "p.cpp").write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-isystem", cuda, str(tmp_path / "p.cpp"), "-o", str(tmp_path / "p")], check=True)
    r = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_operators_between_the_projections_ask_so():
    for name in ("norm.cu", "fp8_block.cu", "rotary.cu"):
        text = open(os.path.join(CSRC, name), encoding="utf-8").read()
        assert not re.search(r"static (std::atomic<)?(int|bool|float)\b[^(;]*;", text), name
        for m in re.finditer(r"cudaOccupancy\w+\(", text):
            assert re.search(r"known\.get\([^;]*$|known\.get\((.|\n)*return $", text[:m.start()][-1500:]), (name, text[m.start():][:60])
