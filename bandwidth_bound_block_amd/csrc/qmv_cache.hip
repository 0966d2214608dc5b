// Writing new keys and values into a quantized cache, and reading slots back.
//
// A thread has an octet of a token's head: four neighbouring threads share a
// block of 32 values and its scale.  Both are bound by memory (a write of 6000
// tokens of 8 heads of 128 from fp32, 60 MB, takes 18 us) and, for a few tokens,
// by the launch (48 tokens 5 us, 333 read 3 us).
#include <algorithm>

#include "qmv_block_decode.h"
#include "qmv_cache.h"

namespace qmv {

int32_t check_cache(const char* name, const qmv_cache* c) {
    if (!c) return fail(QMV_EINVAL, "%s: null pointer", name);
    if (c->k_fmt < QMV_Q8_0 || c->k_fmt > QMV_Q4_1 || c->v_fmt < QMV_Q8_0 || c->v_fmt > QMV_Q4_1)
        return fail(QMV_EUNSUPPORTED, "%s: a cache's format must be Q8_0, Q4_0 or Q4_1", name);
    if (!c->k || !c->v) return fail(QMV_EINVAL, "%s: null pointer", name);
    if (c->n_kv_heads < 1 || c->n_kv_heads > 1024)
        return fail(QMV_EINVAL, "%s: n_kv_heads must be 1..1024", name);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(QMV_EINVAL, "%s: head_dim must be 64, 128 or 256", name);
    if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
        return fail(QMV_EINVAL, "%s: page_size must be a power of two, 16..4096", name);
    if (c->n_pages < 1 || c->n_pages > ((int64_t(1) << 31) - 1) / c->page_size)
        return fail(QMV_EINVAL, "%s: n_pages must be >= 1 with n_pages * page_size < 2^31", name);
    if (c->reserved != 0) return fail(QMV_EINVAL, "%s: reserved must be 0", name);
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return fail(QMV_EALIGN, "%s: a cache's pages must be 16-byte aligned", name);
    return QMV_OK;
}

namespace {

constexpr int kCT = 256;
constexpr float kLimit = 65024.f;    // 127 * 512: scales and values stay within fp16

struct SideArgs {
    CacheSide c;
    const void* x;                   // write: the new values
    int64_t st, sh;
    void* out;                       // read
    bool vec;
};
struct CacheArgs {
    SideArgs side[2];
    const int32_t* slots;
    int64_t n;                       // tokens
    int64_t n_slots;
    int32_t heads, page_shift, oct_shift, nb_shift;    // log2 of octets and of blocks of a row
};

// Lanes of a quad: the value of lane ^ 1 and lane ^ 2.
template <int X>
__device__ __forceinline__ float quad_xor(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), X == 1 ? 0xb1 : 0x4e, 0xf, 0xf, true));
}

// Codes of w for a scale d (and minimum m): those of the exact quotient.  The
// fp32 quotient is at most 2^-14 off where the code is within its range, so
// only next to a border between two codes is the fp64 one needed (its
// rounding, 2^-53, is less than any quotient's distance from a border that it
// is not on: w and d together have 35 bits; with a minimum the difference of w
// and m is rounded to fp64 first).
__device__ __forceinline__ void codes_of(const float (&w)[8], float d, float m, float lo, float hi, int (&c)[8]) {
    const float inv = 1.f / d;
    bool near = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = (w[j] - m) * inv, r = __builtin_rintf(t);
        near |= __builtin_fabsf(__builtin_fabsf(t - r) - 0.5f) < 6.2e-5f;
        c[j] = (int)fminf(fmaxf(r, lo), hi);
    }
    if (near) {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            float v = w[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) v = j == k ? w[k] : v;
            const double t = ((double)v - (double)m) / (double)d;
            const double r = __builtin_copysign(__builtin_floor(__builtin_fabs(t) + 0.5), t);
            const int e = (int)fmin(fmax(r, (double)lo), (double)hi);
#pragma unroll
            for (int k = 0; k < 8; ++k) c[k] = j == k ? e : c[k];
        }
    }
}

template <class XT>
__device__ __forceinline__ void load_octet(const XT* p, bool vec, float (&w)[8]) {
    if (vec) {
        const float4 a = XIn<XT>::load4(p), b = XIn<XT>::load4(p + 4);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = XIn<XT>::load1(p + j);
    }
}

// grid (tokens' octets, heads, keys and values)
template <class XT>
__global__ __launch_bounds__(kCT) void cache_write_kernel(const CacheArgs a) {
    const SideArgs& s = a.side[blockIdx.z];
    const int h = blockIdx.y;
    const int64_t all = a.n << a.oct_shift, step = (int64_t)gridDim.x * kCT;
    for (int64_t i = (int64_t)blockIdx.x * kCT + threadIdx.x; i < all; i += step) {
        const int64_t t = i >> a.oct_shift;
        const int o = (int)(i & ((1 << a.oct_shift) - 1));
        const int64_t slot = a.slots[t];
        if (slot < 0 || slot >= a.n_slots) continue;        // alike for the four lanes of a block
        float w[8];
        load_octet<XT>(static_cast<const XT*>(s.x) + t * s.st + h * s.sh + 8 * o, s.vec, w);
        bool bad = false;
        float amax = 0.f, ext = 0.f, mn = __builtin_inff(), mx = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bad |= !(__builtin_fabsf(w[j]) < __builtin_inff());
            w[j] = fminf(fmaxf(w[j], -kLimit), kLimit);
            if (__builtin_fabsf(w[j]) > amax) {
                amax = __builtin_fabsf(w[j]);
                ext = w[j];
            }
            mn = fminf(mn, w[j]);
            mx = fmaxf(mx, w[j]);
        }
        float nf = bad ? 1.f : 0.f;
        const int lane = threadIdx.x;
#define QMV_MEET(X)                                                                            \
    {                                                                                          \
        const float e = quad_xor<X>(ext), am = __builtin_fabsf(e);                             \
        if (am > amax || (am == amax && (lane & X))) { /* of equal ones the lower lane's */    \
            amax = am;                                                                         \
            ext = e;                                                                           \
        }                                                                                      \
        mn = fminf(mn, quad_xor<X>(mn));                                                       \
        mx = fmaxf(mx, quad_xor<X>(mx));                                                       \
        nf = fmaxf(nf, quad_xor<X>(nf));                                                       \
    }
        QMV_MEET(1)
        QMV_MEET(2)
#undef QMV_MEET
        const int nb = 1 << a.nb_shift, b = o >> 2, g = o & 3, place = (g << a.nb_shift) + b;
        const int64_t page = slot >> a.page_shift;
        const int off = (int)(slot & ((1 << a.page_shift) - 1));
        uint8_t* head = s.c.pages + page * s.c.page_bytes + h * s.c.head_bytes;
        _Float16* scale = reinterpret_cast<_Float16*>(head + ((int64_t)s.c.row << a.page_shift)) + ((b << a.page_shift) + off);
        int c[8];
        _Float16 d, m = (_Float16)0.f;
        if (s.c.fmt == QMV_Q8_0) {
            d = (_Float16)(amax / 127.f);
            if ((float)d != 0.f) codes_of(w, (float)d, 0.f, -127.f, 127.f, c);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] = 0;
            uint2 u;
            u.x = (c[0] & 255) | (c[1] & 255) << 8 | (c[2] & 255) << 16 | c[3] << 24;
            u.y = (c[4] & 255) | (c[5] & 255) << 8 | (c[6] & 255) << 16 | c[7] << 24;
            *reinterpret_cast<uint2*>(head + (int64_t)off * s.c.row + 8 * place) = u;
        } else {
            float bias = 8.f, mf = 0.f;
            if (s.c.fmt == QMV_Q4_0) {
                d = (_Float16)(ext / -8.f) + (_Float16)0.f;      // no -0: the same bytes whichever zero is first
            } else {
                bias = 0.f;
                m = (_Float16)mn + (_Float16)0.f;
                mf = (float)m;
                // two roundings, as for the other formats: the compiler makes one of the two casts
                float q = (float)(((double)mx - (double)mn) / 15.0);
                asm("" : "+v"(q));
                d = (_Float16)q;
            }
            if ((float)d != 0.f) codes_of(w, (float)d, mf, -bias, 15.f - bias, c);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] = 0;
            uint32_t u = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) u |= (uint32_t)(c[j] + (int)bias) << (4 * (j >> 1) + 16 * (j & 1));
            *reinterpret_cast<uint32_t*>(head + (int64_t)off * s.c.row + 4 * place) = u;
        }
        if (g == 0) {
            scale[0] = nf != 0.f ? (_Float16)__builtin_nanf("") : d;
            if (s.c.fmt == QMV_Q4_1) scale[(int64_t)nb << a.page_shift] = m;
        }
    }
}

template <class XT>
__device__ __forceinline__ void store_octet(XT* p, const float (&v)[8]) {
    XT e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = (XT)v[j];
    if constexpr (sizeof(XT) == 4) {
        reinterpret_cast<float4*>(p)[0] = float4{v[0], v[1], v[2], v[3]};
        reinterpret_cast<float4*>(p)[1] = float4{v[4], v[5], v[6], v[7]};
    } else {
        uint4 u;
        __builtin_memcpy(&u, e, 16);
        *reinterpret_cast<uint4*>(p) = u;
    }
}

// The octet o of U heads from h0 on (fewer at the end) of one token: all loads, then all values.
template <int F, class XT, int U>
__device__ __forceinline__ void read_heads(const CacheArgs& a, const SideArgs& s, int64_t t, int o, int64_t slot, int h0) {
    const int b = o >> 2, g = o & 3, place = (g << a.nb_shift) + b;
    const int off = (int)(slot & ((1 << a.page_shift) - 1));
    const uint8_t* page = s.c.pages + (slot >> a.page_shift) * s.c.page_bytes + h0 * s.c.head_bytes;
    const uint32_t code = off * s.c.row + (F == QMV_Q8_0 ? 8 : 4) * place;
    const uint32_t scale = (s.c.row << a.page_shift) + 2 * ((b << a.page_shift) + off), min = scale + (2 << (a.nb_shift + a.page_shift));
    uint32_t w[U][F == QMV_Q8_0 ? 2 : 1];
    uint16_t d[U], m[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const uint8_t* p = page + (U == 1 || h0 + k < a.heads ? k : 0) * s.c.head_bytes;
        if constexpr (F == QMV_Q8_0) {
            const uint2 u = *reinterpret_cast<const uint2*>(p + code);
            w[k][0] = u.x ^ 0x80808080u;
            w[k][1] = u.y ^ 0x80808080u;
        } else {
            w[k][0] = *reinterpret_cast<const uint32_t*>(p + code);
        }
        d[k] = *reinterpret_cast<const uint16_t*>(p + scale);
        m[k] = F == QMV_Q4_1 ? *reinterpret_cast<const uint16_t*>(p + min) : 0;
    }
    XT* out = static_cast<XT*>(s.out) + ((t * a.heads + h0) << a.oct_shift) * 8 + 8 * o;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (U > 1 && h0 + k >= a.heads) break;
        f16x2 c[4];
        if constexpr (F == QMV_Q8_0) {
            c[0] = byte_pair<0, 1>(w[k][0], 0);
            c[1] = byte_pair<2, 3>(w[k][0], 0);
            c[2] = byte_pair<0, 1>(w[k][1], 0);
            c[3] = byte_pair<2, 3>(w[k][1], 0);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = nibble_pair(w[k][0], j, F == QMV_Q4_0 ? 8.f : 0.f);
        }
        const float df = (float)__builtin_bit_cast(_Float16, d[k]), mf = (float)__builtin_bit_cast(_Float16, m[k]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = F == QMV_Q4_1 ? __builtin_fmaf((float)c[j / 2][j & 1], df, mf) : (float)c[j / 2][j & 1] * df;
        store_octet<XT>(out + ((int64_t)k << a.oct_shift) * 8, v);
    }
}

// grid (tokens' octets, U heads, keys and values)
template <class XT, int U>
__global__ __launch_bounds__(kCT) void cache_read_kernel(const CacheArgs a) {
    const SideArgs& s = a.side[blockIdx.z];
    if (!s.out) return;
    const int h0 = blockIdx.y * U;
    const int64_t all = a.n << a.oct_shift, step = (int64_t)gridDim.x * kCT;
    for (int64_t i = (int64_t)blockIdx.x * kCT + threadIdx.x; i < all; i += step) {
        const int64_t t = i >> a.oct_shift;
        const int o = (int)(i & ((1 << a.oct_shift) - 1));
        const int64_t slot = a.slots[t];
        if (slot < 0 || slot >= a.n_slots) {
            const float nan = __builtin_nanf(""), v[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
            for (int h = h0; h < min(h0 + U, a.heads); ++h)
                store_octet<XT>(static_cast<XT*>(s.out) + ((t * a.heads + h) << a.oct_shift) * 8 + 8 * o, v);
        } else if (s.c.fmt == QMV_Q8_0) {
            read_heads<QMV_Q8_0, XT, U>(a, s, t, o, slot, h0);
        } else if (s.c.fmt == QMV_Q4_0) {
            read_heads<QMV_Q4_0, XT, U>(a, s, t, o, slot, h0);
        } else {
            read_heads<QMV_Q4_1, XT, U>(a, s, t, o, slot, h0);
        }
    }
}

CacheArgs cache_args(const qmv_cache& c, const int32_t* slots, int64_t n) {
    CacheArgs a{};
    a.side[0].c = cache_side(c, true);
    a.side[1].c = cache_side(c, false);
    a.slots = slots;
    a.n = n;
    a.n_slots = c.n_pages * c.page_size;
    a.heads = c.n_kv_heads;
    a.page_shift = log2_of(c.page_size);
    a.oct_shift = log2_of(c.head_dim / 8);
    a.nb_shift = log2_of(c.head_dim / 32);
    return a;
}
// Workgroups along the tokens: a launch holds 2^32 threads.
dim3 cache_grid(const CacheArgs& a) {
    const int64_t all = ((a.n << a.oct_shift) + kCT - 1) / kCT;
    return dim3((unsigned)std::min<int64_t>(all, (int64_t(1) << 22) / a.heads), a.heads, 2);
}

// Heads of a thread of the read, which shares the slot's page and the addresses
// between them: four once two workgroups for each compute unit are left.  65536
// tokens of 8 heads of 128: 72 us (344 MB, 4.8 TB/s, what a copy reaches), one
// head a thread 126; 32000 30.0 and 31.6.  To fp32 6000 tokens of Q8_0 and Q4_1
// 14.2 and 16.3, but of Q4_0 8000 21.7 and 17.9, 32000 80 and 77.  Under the
// border (2048 tokens of 8 heads) both are the launch.
constexpr int kReadHeads = 4;
template <class XT>
void launch_read(const CacheArgs& a, hipStream_t st) {
    dim3 grid = cache_grid(a);
    if ((int64_t)grid.x * a.heads >= 512 * kReadHeads) {
        grid.y = (a.heads + kReadHeads - 1) / kReadHeads;
        hipLaunchKernelGGL((cache_read_kernel<XT, kReadHeads>), grid, dim3(kCT), 0, st, a);
    } else {
        hipLaunchKernelGGL((cache_read_kernel<XT, 1>), grid, dim3(kCT), 0, st, a);
    }
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_cache_page_bytes(qmv_fmt fmt, int32_t n_kv_heads, int32_t head_dim, int32_t page_size) {
    if (n_kv_heads < 1 || n_kv_heads > 1024 || (head_dim != 64 && head_dim != 128 && head_dim != 256) || page_size < 16 ||
        page_size > 4096 || (page_size & (page_size - 1)))
        return 0;
    const int block = fmt == QMV_Q8_0 ? 34 : fmt == QMV_Q4_0 ? 18 : fmt == QMV_Q4_1 ? 20 : 0;
    return (size_t)n_kv_heads * page_size * (head_dim / 32) * block;
}

extern "C" int32_t qmv_cache_write(const qmv_cache* cache, const void* k, int64_t k_stride_token, int64_t k_stride_head,
                                   const void* v, int64_t v_stride_token, int64_t v_stride_head, int32_t x_type,
                                   const int32_t* slots, int64_t n_tokens, void* stream) {
    using namespace qmv;
    const char* name = "qmv_cache_write";
    if (const int32_t e = check_cache(name, cache)) return e;
    if (!k || !v || !slots) return fail(QMV_EINVAL, "%s: null pointer", name);
    const int xe = type_bytes(x_type);
    if (!xe) return fail(QMV_EINVAL, "%s: unknown x_type %d", name, (int)x_type);
    if (n_tokens < 1 || n_tokens > (1 << 24)) return fail(QMV_EINVAL, "%s: n_tokens must be 1..2^24", name);
    if (cache->n_kv_heads > 1 && (k_stride_head < cache->head_dim || v_stride_head < cache->head_dim))
        return fail(QMV_EINVAL, "%s: the strides per head must be >= head_dim", name);
    if (!aligned(k, xe) || !aligned(v, xe) || !aligned(slots, 4))
        return fail(QMV_EALIGN, "%s: a pointer is not aligned to its elements", name);
    CacheArgs a = cache_args(*cache, slots, n_tokens);
    const void* x[2] = {k, v};
    const int64_t st[2] = {k_stride_token, v_stride_token}, sh[2] = {k_stride_head, v_stride_head};
    for (int i = 0; i < 2; ++i) {
        a.side[i].x = x[i];
        a.side[i].st = st[i];
        a.side[i].sh = cache->n_kv_heads > 1 ? sh[i] : 0;
        a.side[i].vec = aligned(x[i], 16) && (st[i] * xe) % 16 == 0 && (a.side[i].sh * xe) % 16 == 0;
    }
    const dim3 grid = cache_grid(a);
    const hipStream_t s = as_stream(stream);
    switch (x_type) {
    case QMV_X_F32: hipLaunchKernelGGL((cache_write_kernel<float>), grid, dim3(kCT), 0, s, a); break;
    case QMV_X_F16: hipLaunchKernelGGL((cache_write_kernel<_Float16>), grid, dim3(kCT), 0, s, a); break;
    default: hipLaunchKernelGGL((cache_write_kernel<__bf16>), grid, dim3(kCT), 0, s, a); break;
    }
    return check_launch(name);
}

extern "C" int32_t qmv_cache_read(const qmv_cache* cache, const int32_t* slots, int64_t n_tokens, void* k_out, void* v_out,
                                  int32_t out_type, void* stream) {
    using namespace qmv;
    const char* name = "qmv_cache_read";
    if (const int32_t e = check_cache(name, cache)) return e;
    if (!slots || (!k_out && !v_out)) return fail(QMV_EINVAL, "%s: null pointer", name);
    if (!type_bytes(out_type)) return fail(QMV_EINVAL, "%s: unknown out_type %d", name, (int)out_type);
    if (n_tokens < 1 || n_tokens > (1 << 24)) return fail(QMV_EINVAL, "%s: n_tokens must be 1..2^24", name);
    if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return fail(QMV_EALIGN, "%s: the outputs must be 16-byte aligned, slots 4-byte", name);
    CacheArgs a = cache_args(*cache, slots, n_tokens);
    a.side[0].out = k_out;
    a.side[1].out = v_out;
    const hipStream_t s = as_stream(stream);
    switch (out_type) {
    case QMV_X_F32: launch_read<float>(a, s); break;
    case QMV_X_F16: launch_read<_Float16>(a, s); break;
    default: launch_read<__bf16>(a, s); break;
    }
    return check_launch(name);
}
