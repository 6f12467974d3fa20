// Rows of channels in registers, shared by the residual join, the layer norm, the
// lookup and the weighted sum (gfx950): 16-byte chunks of a row and sums over the
// lanes that hold one.
#pragma once

#include "zs_internal.h"
#include "zs_tile.h"

namespace zs {

template <typename T>
struct Chunk {
    static constexpr int V = 16 / sizeof(T);
    __device__ static void unpack(u32x4 raw, float (&f)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bits = raw[i];
                f[i] = __builtin_bit_cast(float, bits);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __builtin_bit_cast(float, raw[i] << 16);
                f[2 * i + 1] = __builtin_bit_cast(float, raw[i] & 0xffff0000u);
            }
        }
    }
    __device__ static u32x4 pack(const float (&f)[V]) {
        union {
            T e[V];
            u32x4 v;
        } u;
#pragma unroll
        for (int i = 0; i < V; ++i) u.e[i] = T(f[i]);
        return u.v;
    }
};

// Chunk `chunk` of a row of c elements (zeros outside).  vec: whole chunks on 16
// bytes; NT: read once, past the caches.
template <typename T, bool NT = false>
__device__ inline u32x4 load_chunk(const T* row, int chunk, int c, bool vec) {
    constexpr int V = Chunk<T>::V;
    const int left = c - chunk * V;
    if (NT && vec)
        return left > 0
                   ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + chunk * V))
                   : u32x4{0, 0, 0, 0};
    if (vec) return left > 0 ? *reinterpret_cast<const u32x4*>(row + chunk * V) : u32x4{0, 0, 0, 0};
    return load_partial(row + chunk * V, left);
}
template <typename T>
__device__ inline void store_chunk(T* row, int chunk, int c, bool vec, u32x4 v,
                                   bool stream = false) {
    constexpr int V = Chunk<T>::V;
    const int left = c - chunk * V;
    if (vec && stream) {
        if (left > 0) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(row + chunk * V));
        return;
    }
    if (vec) {
        if (left > 0) *reinterpret_cast<u32x4*>(row + chunk * V) = v;
        return;
    }
    union {
        u32x4 v;
        T e[V];
    } u;
    u.v = v;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < left) row[chunk * V + i] = u.e[i];
}
// The same for rows that may start and end anywhere.  A row's last chunk is loaded as the
// row's last 16 bytes (load_raw) and moved down in the registers where it is used
// (settled), and stored in up to three pieces: element by element, the lanes that hold a
// row's end took three times the others' time (layer norm's gradients of 248406 x 95 in
// bf16 105 us, 44 so).  Moved down where it is loaded, each load would be waited for before
// the next is asked for, in rows of whole chunks too where one kernel serves both (lookup of
// 65536 rows of 1024 in bf16 44 us against 33.5, sum of 31837 x 2 x 831 in fp32 77 against 64).
template <typename T>
__device__ inline u32x4 move_down(u32x4 v, int elements) {
    constexpr int word = 4 / sizeof(T);   // elements of one
    if (elements & (2 * word)) v = u32x4{v[2], v[3], 0, 0};
    if (elements & word) v = u32x4{v[1], v[2], v[3], 0};
    if constexpr (word == 2) {
        if (elements & 1)
            v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16,
                      v[3] >> 16};
    }
    return v;
}
template <typename T, bool NT = false>
__device__ inline u32x4 load_raw(const T* row, int chunk, int c, bool vec) {
    constexpr int V = Chunk<T>::V;
    if (vec) return load_chunk<T, NT>(row, chunk, c, true);
    if (c < V) return load_partial(row, chunk == 0 ? c : 0);   // the row is less than a chunk
    if (chunk * V >= c) return u32x4{0, 0, 0, 0};
    const int at = chunk * V < c - V ? chunk * V : c - V;
    u32x4 v;
    __builtin_memcpy(&v, row + at, 16);
    return v;
}
template <typename T>
__device__ inline u32x4 settled(u32x4 v, int chunk, int c, bool vec) {
    constexpr int V = Chunk<T>::V;
    const int back = (chunk + 1) * V - c;
    if (vec || c < V || back <= 0) return v;
    return back < V ? move_down<T>(v, back) : u32x4{0, 0, 0, 0};
}
template <typename T>
__device__ inline void store_any(T* row, int chunk, int c, bool vec, u32x4 v) {
    constexpr int V = Chunk<T>::V;
    if (vec) return store_chunk(row, chunk, c, true, v);
    const int left = c - chunk * V;
    T* at = row + chunk * V;
    if (left >= V) {
        __builtin_memcpy(at, &v, 16);
        return;
    }
    if (left <= 0) return;
    constexpr int word = 4 / sizeof(T);
    if (left & (2 * word)) {
        const u32x2 low = {v[0], v[1]};
        __builtin_memcpy(at, &low, 8);
        at += 2 * word, v = u32x4{v[2], v[3], 0, 0};
    }
    if (left & word) {
        const uint32_t low = v[0];
        __builtin_memcpy(at, &low, 4);
        at += word, v[0] = v[1];
    }
    if constexpr (word == 2) {
        if (left & 1) {
            const uint16_t low = uint16_t(v[0]);
            __builtin_memcpy(at, &low, 2);
        }
    }
}
// V fp32 parameters of a chunk.
template <int V>
__device__ inline void load_param(const float* p, int chunk, int c, bool vec, float (&f)[V]) {
    const int left = c - chunk * V;
    if (vec) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4 t = left > 0 ? *reinterpret_cast<const f32x4*>(p + chunk * V + i)
                                     : f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) f[i + q] = t[q];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i < left ? p[chunk * V + i] : 0.0f;
    }
}

// v of the lane that a DPP control picks within 16 lanes.
template <int CTRL>
__device__ inline float dpp(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// Sum over the L <= 64 lanes of a row, in all of them, without LDS: halves are
// exchanged within 16 lanes by DPP (xor 1, xor 2, mirrors of 8 and 16 lanes),
// then across 16 and 32 lanes by the permlane swaps, whose two results are the
// two halves.
template <int L>
__device__ inline float lane_sum(float v) {
    if constexpr (L >= 2) v += dpp<0xB1>(v);
    if constexpr (L >= 4) v += dpp<0x4E>(v);
    if constexpr (L >= 8) v += dpp<0x141>(v);
    if constexpr (L >= 16) v += dpp<0x140>(v);
    if constexpr (L >= 32) {
        const int i = __builtin_bit_cast(int, v);
        const auto r = __builtin_amdgcn_permlane16_swap(i, i, false, false);
        const uint32_t a = r[0], b = r[1];
        v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    }
    if constexpr (L >= 64) {
        const int i = __builtin_bit_cast(int, v);
        const auto r = __builtin_amdgcn_permlane32_swap(i, i, false, false);
        const uint32_t a = r[0], b = r[1];
        v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    }
    return v;
}

// Sums of N values over the L lanes of a row.  Above a wavefront the row is the
// workgroup's and the wavefronts meet in LDS: `region` alternates, so that one
// barrier per sum is enough (a region is written again only behind the next
// sum's barrier).
template <int L, int N>
__device__ inline void row_sum(float (&v)[N], float* lds, int& region) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_sum<(L < 64 ? L : 64)>(v[i]);
    if constexpr (L > 64) {
        constexpr int W = L / 64;
        float* at = lds + region * W * 2;
        region ^= 1;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) at[wave * 2 + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += at[w * 2 + i];
            v[i] = s;
        }
    }
}

}  // namespace zs
