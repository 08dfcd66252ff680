"""What the forward norms read of gamma and beta at widths that are no whole number of vectors: every
element of the row's columns, and nothing outside the parameter. The kernels' own rule (rmsq_param.h)
runs here against a reader that checks each access, for every width, shift and column vector."""
import pytest

import host_program

PROGRAM = """
#include <cstdio>
#include <vector>
#include "rmsq_param.h"

// element i holds i + 1 (16 bits: in 16 bits)
template <int VW> struct Checked {
    int hidden;
    long* outside;
    void read(int k) const { if (k < 0 || k >= hidden) ++*outside; }
    uint32_t element(int k) const { read(k); return static_cast<uint32_t>(k + 1); }
    void vector(int k, uint32_t* w) const
    {
        if (k % VW != 0) ++*outside;
        for (int j = 0; j < 4; ++j) w[j] = 0;
        for (int j = 0; j < VW; ++j) w[j * 4 / VW] |= element(k + j) << (VW == 8 ? 16 * (j & 1) : 0);
    }
};

template <int VW> void sweep(int first, int last, long* outside, long* wrong, long* vectors)
{
    for (int hidden = first; hidden <= last; ++hidden) {
        if (hidden % VW == 0) continue;
        for (int shift = 0; shift < VW; ++shift) {
            // the shifts that rows of this width have
            bool some = false;
            for (int row = 0; row < VW; ++row) some = some || static_cast<long>(row) * hidden % VW == shift;
            for (int k = 0; some && k < shift + hidden; k += VW) {
                uint32_t v[4];
                rmsq::param_words<VW>(Checked<VW>{hidden, outside}, k, shift, hidden, v);
                ++*vectors;
                for (int j = 0; j < VW; ++j) {
                    const int e = k + j - shift;
                    if (e < 0 || e >= hidden) continue;
                    const uint32_t got = VW == 8 ? (v[j / 2] >> (16 * (j & 1))) & 0xFFFFu : v[j];
                    if (got != static_cast<uint32_t>(e + 1)) ++*wrong;
                }
            }
        }
    }
}

int main()
{
    long outside = 0, wrong = 0, vectors = 0;
    sweep<VECTOR>(FIRST, LAST, &outside, &wrong, &vectors);
    std::printf("%ld outside, %ld wrong, %d\\n", outside, wrong, vectors > 0);
}
"""


@pytest.mark.parametrize("vector", [8, 4])
@pytest.mark.parametrize("first,last", [(1, 300), (1003, 1003), (2051, 2053), (5121, 5125), (32761, 32767), (65529, 65535)])
def test_nothing_outside_the_parameter_is_read(vector, first, last, tmp_path):
    program = PROGRAM.replace("VECTOR", str(vector)).replace("FIRST", str(first)).replace("LAST", str(last))
    out = host_program.run(program, tmp_path)
    assert out.strip() == "0 outside, 0 wrong, 1"
