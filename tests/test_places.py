"""What the checks of arguments know of the memory that strided tensors take, against every byte of small ones."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <random>
#include <set>

#include "places.h"
using namespace dbs::ops;

int main()
{
    std::mt19937 g(5);
    auto in = [&](int a, int b) { return a + (int)(g() % (unsigned)(b - a + 1)); };
    long wrong = 0, missed = 0, taken_for_own = 0, own_missed = 0, meet = 0;
    for (int it = 0; it < 100000; ++it) {
        // any strides, or (nested) parts cut out of one buffer [a][b][h][d]
        const bool nested = it % 2;
        const int d = in(1, 4), H = in(1, 6), B = in(1, 4), A = in(1, 3);
        int at[2], run[2], count[2][3], stride[2][3];
        std::set<int> bytes[2];
        bool twice[2] = {false, false};
        for (int q = 0; q < 2; ++q) {
            if (nested) {
                const int a0 = in(0, A - 1), b0 = in(0, B - 1), h0 = in(0, H - 1);
                run[q] = in(1, d);
                const int s[3] = {d * H * B, d * H, d}, c[3] = {in(1, A - a0), in(1, B - b0), in(1, H - h0)};
                at[q] = 1000 + a0 * s[0] + b0 * s[1] + h0 * s[2] + in(0, d - run[q]);
                for (int i = 0; i < 3; ++i) stride[q][i] = s[i], count[q][i] = c[i];
            } else {
                at[q] = 1000 + in(0, 40);
                run[q] = in(1, 5);
                for (int i = 0; i < 3; ++i) stride[q][i] = in(0, 20), count[q][i] = in(1, 4);
            }
            for (int x = 0; x < count[q][0]; ++x)
                for (int y = 0; y < count[q][1]; ++y)
                    for (int z = 0; z < count[q][2]; ++z)
                        for (int r = 0; r < run[q]; ++r)
                            twice[q] |= !bytes[q].insert(at[q] + x * stride[q][0] + y * stride[q][1] + z * stride[q][2] + r).second;
        }
        Places p[2];
        for (int q = 0; q < 2; ++q)
            p[q] = {(void *)(intptr_t)at[q], 1, run[q], {{count[q][0], stride[q][0]}, {count[q][1], stride[q][1]}, {count[q][2], stride[q][2]}}};
        bool shared = false;
        for (int x : bytes[0]) shared |= bytes[1].count(x) > 0;
        for (int q = 0; q < 2; ++q) {
            const bool said = p[q].meets(p[1 - q]);
            wrong += said && !shared;
            missed += !said && shared;
            taken_for_own += p[q].own && twice[q];
            own_missed += nested && !p[q].own;
        }
        meet += shared;
    }
    std::printf("%ld %ld %ld %ld %d\n", wrong, missed, taken_for_own, own_missed, meet > 10000);
    const Places none((void *)1000, 2, 64, {{0, 64}, {3, 0}}), some((void *)1000, 2, 64, {{4, 64}});
    std::printf("%d %d %d %d\n", none.own, none.meets(some), some.meets(none), some.same(some));
}
"""


def test_places_against_every_byte(tmp_path):
    src, exe = tmp_path / "places.cpp", tmp_path / "places"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "dynamic_sparsity_spmspv_gb300", "csrc"), "-o", str(exe), str(src)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120).stdout.split("\n")
    assert out[0].split() == ["0", "0", "0", "0", "1"] and out[1].split() == ["1", "0", "0", "1"]
