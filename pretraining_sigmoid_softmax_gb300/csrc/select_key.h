// The integer keys of the choice of experts: a value in [0, 1) as a 23-bit fixed-point number above
// the expert's index.
#pragma once

#include <limits.h>
#include <stdint.h>

#ifdef __CUDACC__
#define MOE_KEY_FN __host__ __device__ __forceinline__
#else
#define MOE_KEY_FN inline
#endif

namespace moe {

constexpr int kKeyBits = 9;
constexpr float kUnits = 8388608.f;  // per 1

// From the bits of v + 1, whose mantissa is v's fixed-point number: shifted left they are the key's
// upper bits (sign and exponent, 127, leave the word), in unsigned arithmetic, which wraps, turned so
// that signed integers order the keys. `id` = expert + 1 + INT_MIN, so that INT_MIN is no expert's
// key.
MOE_KEY_FN int key_of(uint32_t bits, int id) {
    return (int)((bits << kKeyBits) + (uint32_t)id);
}
MOE_KEY_FN int expert_of(int key) { return (key & ((1 << kKeyBits) - 1)) - 1; }
MOE_KEY_FN int units_of(int key) { return (int)((uint32_t)(key ^ INT_MIN) >> kKeyBits); }

}  // namespace moe
