// ls_elements.hpp -- float32, float16 and bfloat16 elements in 32-bit words (gfx950).
// Arithmetic is in float32; pack rounds once, to nearest, ties to even.
#pragma once
#include "ls_device.hpp"

namespace ls {

// unpack / pack: the one or two elements of a word (one 16-bit element: its low half).
struct F32 {
    static constexpr int size = 4;
    static __device__ __forceinline__ void unpack(uint32_t w, float (&v)[1]) { v[0] = from_bits<float>(w); }
    static __device__ __forceinline__ uint32_t pack(const float (&v)[1]) { return to_bits(v[0]); }
};
struct F16 {
    static constexpr int size = 2;
    typedef _Float16 x2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ void unpack(uint32_t w, float (&v)[2])
    {
        const x2 h = __builtin_bit_cast(x2, w);
        v[0] = float(h.x);
        v[1] = float(h.y);
    }
    static __device__ __forceinline__ void unpack(uint32_t w, float (&v)[1])
    {
        v[0] = float(__builtin_bit_cast(x2, w).x);
    }
    template <int N>
    static __device__ __forceinline__ uint32_t pack(const float (&v)[N])
    {
        x2 h;
        h.x = static_cast<_Float16>(v[0]);
        h.y = static_cast<_Float16>(v[N - 1]);
        return __builtin_bit_cast(uint32_t, h);
    }
};
struct BF16 {
    static constexpr int size = 2;
    typedef __bf16 x2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ void unpack(uint32_t w, float (&v)[2])
    {
        v[0] = from_bits<float>(w << 16);
        v[1] = from_bits<float>(w & 0xffff0000u);
    }
    static __device__ __forceinline__ void unpack(uint32_t w, float (&v)[1]) { v[0] = from_bits<float>(w << 16); }
    template <int N>
    static __device__ __forceinline__ uint32_t pack(const float (&v)[N])
    {
        x2 h;
        h.x = static_cast<__bf16>(v[0]);
        h.y = static_cast<__bf16>(v[N - 1]);
        return __builtin_bit_cast(uint32_t, h);
    }
};

// VEC neighbouring elements at p, aligned to all of them or to 16 bytes (eight float32 values are 32 bytes; a
// vector type's own alignment, its size, would promise the compiler more than the launchers ask for).
template <class E, int VEC>
struct Elements {
    static constexpr int per_word = VEC == 1 ? 1 : 4 / E::size;
    static constexpr int words = VEC / per_word;
    static constexpr int align = words < 4 ? 4 * words : 16;
    uint32_t w[words];
    // once: the bytes are not asked for again soon, and need no place in the caches
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const void* p)
    {
        if constexpr (VEC * E::size == 2) {
            w[0] = *static_cast<const uint16_t*>(p);
        } else {
            typedef uint32_t v __attribute__((ext_vector_type(words), aligned(align)));
            v t;
            if constexpr (ONCE)
                t = __builtin_nontemporal_load(static_cast<const v*>(p));
            else
                t = *static_cast<const v*>(p);
            __builtin_memcpy(w, &t, sizeof w);
        }
    }
    template <bool ONCE = false>
    __device__ __forceinline__ void store(void* p) const
    {
        if constexpr (VEC * E::size == 2) {
            *static_cast<uint16_t*>(p) = uint16_t(w[0]);
        } else {
            typedef uint32_t v __attribute__((ext_vector_type(words), aligned(align)));
            v t;
            __builtin_memcpy(&t, w, sizeof w);
            if constexpr (ONCE)
                __builtin_nontemporal_store(t, static_cast<v*>(p));
            else
                *static_cast<v*>(p) = t;
        }
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const
    {
#pragma unroll
        for (int i = 0; i < words; ++i) {
            float t[per_word];
            E::unpack(w[i], t);
#pragma unroll
            for (int k = 0; k < per_word; ++k)
                f[i * per_word + k] = t[k];
        }
    }
    __device__ __forceinline__ void set(const float (&f)[VEC])
    {
#pragma unroll
        for (int i = 0; i < words; ++i) {
            float t[per_word];
#pragma unroll
            for (int k = 0; k < per_word; ++k)
                t[k] = f[i * per_word + k];
            w[i] = E::pack(t);
        }
    }
};

}  // namespace ls
