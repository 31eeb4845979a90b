"""Parts of the norm's kernels by themselves, in small programs of their own."""
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def run(tmp_path, source):
    """Compiles a program against the library's own headers and the library, and returns what it prints."""
    from rl_fine_tuning_gb300 import build
    lib = build.build()
    src, exe = tmp_path / "p.cu", tmp_path / "p"
    src.write_text(source)
    subprocess.check_call([build.nvcc(), *build.ARCH, *build.FLAGS, str(src), "-o", str(exe), lib])
    return subprocess.check_output([str(exe)], text=True, timeout=60,
                                   env={**os.environ, "LD_LIBRARY_PATH": os.path.dirname(lib)}).split()


def test_the_reciprocal_of_every_scale(tmp_path):
    """Each bf16 number from 2^-126 to 2^121, the scales of a checkpoint: the correctly rounded 1 / scale.  (In 64 bits 1 / s of an
    8-bit s lies at least 2^-33 of itself from where fp32 rounds the other way, so that rounding it again changes nothing.)"""
    out = run(tmp_path, '''#include <cstdio>
#include <cstring>
#include "norm_device.cuh"
using namespace grpo;
constexpr int kFirst = 0x0080, kLast = 0x7c00, kN = kLast - kFirst + 1;
__global__ void k(float* r) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < kN) r[i] = scale_reciprocal(bf16_value(kFirst + i));
}
int main() {
    static float r[kN];
    float* dev;
    if (cudaMalloc(&dev, sizeof(r)) != cudaSuccess) return 1;
    k<<<(kN + 255) / 256, 256>>>(dev);
    if (cudaMemcpy(r, dev, sizeof(r), cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
    int bad = 0;
    for (int i = 0; i < kN; ++i) {
        const uint32_t bits = uint32_t(kFirst + i) << 16;
        float s;
        memcpy(&s, &bits, 4);
        bad += r[i] != float(1.0 / double(s));
    }
    printf("%d %d", kN, bad);
    return 0;
}
''')
    assert out == [str(0x7c00 - 0x80 + 1), "0"]


def test_a_wait_that_ran_out_is_not_an_overflow(tmp_path):
    """What the blocks leave (0: nothing, 1: a value that is not finite, 2: a wait that ran out of time) and a sum of dw that is not
    finite, joined: found_inf is the largest."""
    out = run(tmp_path, '''#include <cstdio>
#include "norm.h"
using namespace grpo;
int main() {
    constexpr int kD = 64, kParts = 700;
    static float part[kParts * kD];
    static int bad[kParts];
    NormParams p = {};
    p.d = kD;
    p.weight_f32 = 1;
    if (cudaMalloc(&p.part, sizeof(part)) != cudaSuccess || cudaMalloc(&p.bad, sizeof(bad)) != cudaSuccess ||
        cudaMalloc(&p.found_inf, 4) != cudaSuccess)
        return 1;
    float* dw;
    if (cudaMalloc(&dw, kD * 4) != cudaSuccess) return 1;
    for (int parts : {1, 3, 600, kParts})
        for (int flags = 0; flags < 4; ++flags)          // of the parts: bit 0: a 1, bit 1: a 2
            for (int inf = 0; inf < 3; ++inf) {          // dw: finite, not finite, left out
                for (int i = 0; i < kParts; ++i) bad[i] = 0;
                for (int i = 0; i < kParts * kD; ++i) part[i] = 1.f;
                if (flags & 1) bad[0] = 1;
                if (flags & 2) bad[parts - 1] = 2;
                if (inf == 1) part[7] = 1.f / 0.f;
                int found = 0;
                p.parts = parts;
                p.dweight = inf == 2 ? nullptr : dw;
                cudaMemcpy(p.part, part, sizeof(part), cudaMemcpyHostToDevice);
                cudaMemcpy(p.bad, bad, sizeof(bad), cudaMemcpyHostToDevice);
                cudaMemcpy(p.found_inf, &found, 4, cudaMemcpyHostToDevice);
                if (launch_norm_join(p, true, nullptr) != cudaSuccess) return 2;
                if (cudaMemcpy(&found, p.found_inf, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return 3;
                const int want = flags & 2 ? 2 : (flags & 1) || inf == 1;
                if (found != want) printf("parts %d flags %d inf %d: %d, not %d\\n", parts, flags, inf, found, want);
            }
    printf("done");
    return 0;
}
''')
    assert out == ["done"]
