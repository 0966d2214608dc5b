// The paged key/value cache (layout in qmv.h): host checks and the device
// side's view of a page.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "qmv_host.h"

namespace qmv {

// QMV_OK, or the code of the first thing wrong with a cache.
int32_t check_cache(const char* name, const qmv_cache* c);
// fp32, fp16 or bf16: bytes of an element, 0 for an unknown type.
inline int type_bytes(int32_t t) { return t == QMV_X_F32 ? 4 : t == QMV_X_F16 || t == QMV_X_BF16 ? 2 : 0; }

// One side (keys or values) of a cache.
struct CacheSide {
    uint8_t* pages;
    int64_t page_bytes;
    int64_t head_bytes;    // of a head's part of a page
    int32_t fmt;
    int32_t row;           // bytes of a token's codes
};
inline CacheSide cache_side(const qmv_cache& c, bool keys) {
    const int32_t fmt = keys ? c.k_fmt : c.v_fmt;
    CacheSide s;
    s.pages = static_cast<uint8_t*>(keys ? c.k : c.v);
    s.page_bytes = (int64_t)qmv_cache_page_bytes((qmv_fmt)fmt, c.n_kv_heads, c.head_dim, c.page_size);
    s.head_bytes = s.page_bytes / c.n_kv_heads;
    s.fmt = fmt;
    s.row = fmt == QMV_Q8_0 ? c.head_dim : c.head_dim / 2;
    return s;
}
inline int log2_of(int32_t v) { return 31 - __builtin_clz((unsigned)v); }

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f16x2 as_h2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }
__device__ __forceinline__ uint32_t as_u(f16x2 h) { return __builtin_bit_cast(uint32_t, h); }
__device__ __forceinline__ f16x2 h2(float v) { return f16x2{(_Float16)v, (_Float16)v}; }

// Codes as exact fp16 integers.  1024 + c has c in its lowest mantissa bits.
// The pair (values 2 j, 2 j + 1) of an octet of 4-bit codes, less `bias`.  Mask
// and base from registers: one instruction takes both, which two constants do not.
__device__ __forceinline__ f16x2 nibble_pair(uint32_t w, int j, float bias) {
    uint32_t mask = 0x000f000fu, base = 0x64006400u;
    asm("" : "+s"(mask));
    asm("" : "+v"(base));
    return as_h2(((w >> (4 * j)) & mask) | base) - h2(1024.f + bias);
}
// Bytes lo and hi (0..3 of a, 4..7 of b) of signed codes, which the caller
// has flipped to s + 128.
template <int LO, int HI>
__device__ __forceinline__ f16x2 byte_pair(uint32_t a, uint32_t b) {
    constexpr uint32_t sel = 0x0c000c00u | (HI << 16) | LO;
    return as_h2(__builtin_amdgcn_perm(b, a, sel) | 0x64006400u) - h2(1024.f + 128.f);
}

}  // namespace
}  // namespace qmv
