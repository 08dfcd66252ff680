// rmsq_param.h -- which words of gamma and beta a row's vectors take where rows start off 16-byte
// boundaries. Plain C++, so that a test on the host can run it against a reader that checks every access.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define RMSQ_PARAM_FN __device__ __forceinline__
#else
#define RMSQ_PARAM_FN inline
#endif

namespace rmsq {

// A parameter's elements for the vector at column k of a row with the given shift: elements k - shift on,
// taken out of the two aligned vectors they lie in, as raw words v. Elements outside 0 to hidden are any
// value, but none is read: the row's last column vector can start behind the parameter's end, and then it
// is the lower vector that ends with it. So a vector is read whole only where it ends within hidden, and
// of the two at most one is cut: the upper where k <= hidden, else the lower (the upper is then all
// outside). VW: elements per vector, 8 of 16 bits or 4 of 32. Reader: vector(k, w) reads the four words at
// element k, a multiple of VW; element(k) reads one. shift is the same for the whole row, so the branches
// on it are uniform.
template <int VW, class Reader>
RMSQ_PARAM_FN void param_words(const Reader& p, int k, int shift, int hidden, uint32_t (&out)[4])
{
    uint32_t w[9];
    for (int j = 0; j < 9; ++j) w[j] = 0;
    if (shift > 0 && k >= VW && k <= hidden) p.vector(k - VW, w);
    if (k + VW <= hidden) {
        p.vector(k, w + 4);
    } else {
        const bool past = k > hidden;
        const int first = past ? k - VW : k;
        uint32_t cut[4] = {0, 0, 0, 0};
        for (int j = 0; j < VW; ++j)
            if (first + j < hidden) cut[j * 4 / VW] |= p.element(first + j) << (VW == 8 ? 16 * (j & 1) : 0);
        for (int j = 0; j < 4; ++j) {
            w[j] = past ? cut[j] : w[j];
            w[4 + j] = past ? 0 : cut[j];
        }
    }
    // the vector starts (VW - shift) elements into lower, upper: words first, then half a word
    const int words = VW == 4 ? 4 - shift : 4 - (shift + 1) / 2;
    uint32_t v[5];
    switch (words) {
    case 0:
        for (int j = 0; j < 5; ++j) v[j] = w[j];
        break;
    case 1:
        for (int j = 0; j < 5; ++j) v[j] = w[j + 1];
        break;
    case 2:
        for (int j = 0; j < 5; ++j) v[j] = w[j + 2];
        break;
    case 3:
        for (int j = 0; j < 5; ++j) v[j] = w[j + 3];
        break;
    default:
        for (int j = 0; j < 5; ++j) v[j] = w[j + 4];
    }
    const bool half = VW == 8 && (shift & 1);
    for (int j = 0; j < 4; ++j) out[j] = half ? v[j] >> 16 | v[j + 1] << 16 : v[j];
}

}  // namespace rmsq
