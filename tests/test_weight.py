"""The 64-bit fixed-point softmax weights (csrc/weight.cuh) compiled for the
host and compared with long double exponentials: relative error below 2^-37
where a weight has the digits, half a unit (and 2^-37) where it has not."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r'''
#include "weight.cuh"
#include <cstdio>
#include <cstdlib>
using namespace dlm;
int main() {
    srand48(7);
    const float temps[] = {1.f, 0.7f, 0.2f, 1.3f, 0.1f, 3.f, 1e-4f};
    double worst = 0;
    for (long i = 0; i < 3000000; ++i) {
        const float T = temps[i % 7], m = (float)(drand48() * 40 - 15);
        float z = m - (float)(drand48() * (i % 3 ? 32 : 0.01)) * T;
        if (i % 5 == 0) z = (float)((int)(z * 16) / 16.0);
        if (z > m) z = m;
        const WeightScale s = weight_scale(m, T);
        const long double e = expl(((long double)z - (long double)m) / (long double)T) * 17592186044416.0L;
        const double off = (double)fabsl((long double)weight44(z, s) - e) - 0.5;
        if (off > 0) worst = fmax(worst, off / (double)(e > 1 ? e : 1));
    }
    const WeightScale s = weight_scale(3.f, 1.f);
    bool cut;
    int bad = worst > 7.3e-12;
    bad |= weight44(3.f, s) != (1ull << 44) || weight44(-INFINITY, s) != 0 || weight44(NAN, s) != 0;
    bad |= weight44(-3.4e38f, s) != 0;
    bad |= scale_floor(1000003ull << 40, 0.25f, cut) != (1000003ull << 38) || cut;
    bad |= scale_floor(7, 0.5f, cut) != 3 || !cut || scale_ceil(7, 0.5f) != 4 || scale_ceil(8, 0.5f) != 4;
    bad |= scale_floor(~0ull, 0.99999994f, cut) != 18446742974197923839ull;
    bad |= scale_floor(~0ull, 1e-40f, cut) != 0 || !cut || scale_floor(~0ull, 0.f, cut) != 0 || cut;
    bad |= scale_floor(1ull << 63, 5.421010862427522e-20f, cut) != 0 || scale_ceil(1ull << 63, 5.421010862427522e-20f) != 1;
    printf("worst %.3g\n", worst);
    return bad;
}
'''


@pytest.mark.parametrize("flags", [[], ["-ffp-contract=off"]])
def test_weights_against_long_double(tmp_path, flags):
    src = tmp_path / "w.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "w"
    subprocess.run(["g++", "-O1", "-std=c++17", *flags, "-I", os.path.join(ROOT, "diffusion_decoding_token_gb300", "csrc"),
                    "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


LOG_PROGRAM = r'''
#include "weight.cuh"
#include <cstdio>
#include <cstdlib>
using namespace dlm;
int main() {
    srand48(3);
    long double worst = 0;
    auto look = [&](float x) { worst = fmaxl(worst, fabsl((long double)log_exact(x) - logl((long double)x))); };
    for (int e = -126; e <= 127; ++e)
        for (int i = 0; i < 2000; ++i) look(ldexpf(1.0f + (float)drand48() * (1.0f - 0x1p-23f), e));
    for (int e = -126; e <= 127; ++e) look(ldexpf(1.0f, e)), look(ldexpf(1.0f + 0x1p-23f, e)), look(ldexpf(2.0f - 0x1p-23f, e));
    printf("worst %.3Lg\n", worst);
    return worst > 0x1p-36L || log_exact(1.0f) != 0.0;
}
'''


@pytest.mark.parametrize("flags", [[], ["-ffp-contract=off"]])
def test_logarithm_against_long_double(tmp_path, flags):
    # the row's sums and their quotients: any normal float
    src = tmp_path / "l.cpp"
    src.write_text(LOG_PROGRAM)
    exe = tmp_path / "l"
    subprocess.run(["g++", "-O1", "-std=c++17", *flags, "-I", os.path.join(ROOT, "diffusion_decoding_token_gb300", "csrc"),
                    "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
