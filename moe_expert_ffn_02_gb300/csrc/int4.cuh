// Device code that the two forms of the 4-bit products share: the table of
// an experts call's units, the widening of codes, small copies.
#pragma once
#include "experts_internal.cuh"

namespace moe {
namespace i4 {

// Eight codes of a word, less the zero point, as four bf16 pairs in channel order.  0x4300 | c is
// 128 + c in bf16, which has 8 significant bits; less 128 + z it is c - z, exactly.
__device__ __forceinline__ void widen(uint32_t word, uint32_t zz, uint32_t (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v;
        asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)));     // (a & b) | c
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                         *reinterpret_cast<const __nv_bfloat162*>(&zz));
        out[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {       // the rest of the 16 is zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ int group_of(const Int4Call& c, int step32) {
    return c.group_inv ? (int)__umulhi((uint32_t)step32, c.group_inv) : step32;
}

// Row tiles per expert as prefix sums: start[e] row tiles of `tile_rows` rows lie before expert e's, whose
// first row is first[e].  Offsets are cut to [0, rows], and one that falls to the largest before it.  Called by the whole CTA; without
// offsets there is nothing to make.
template <int THREADS>
__device__ void row_tiles(const Int4Call& c, int tile_rows, int* start, int* first) {
    __shared__ int sums[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!c.offsets) return;
    bool bad = false;
    for (int e = threadIdx.x; e <= c.E; e += THREADS) {
        const int v = c.offsets[e], cut = min(max(v, 0), c.rows);
        bad |= v != cut;
        first[e] = cut;
    }
    __syncthreads();
    const int per = (c.E + THREADS - 1) / THREADS, e0 = min(c.E, (int)threadIdx.x * per), e1 = min(c.E, e0 + per);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
        const int n = first[e + 1] - first[e];
        bad |= n < 0;
        mine += (max(n, 0) + tile_rows - 1) / tile_rows;
    }
    if (bad && blockIdx.x == 0) atomicOr(c.status, MOE_DEV_BAD_ROW);
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) sums[warp] = incl;
    // Offsets that were cut or fall: one thread makes them rise, so that no row has two experts and there are never
    // more tiles than rows / tile_rows + E, the number that grids and 32-bit counts are made for.
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) {
            int at = 0, low = first[0];
            for (int e = 0; e < c.E; ++e) {
                const int next = max(low, first[e + 1]);
                start[e] = at;
                at += (next - low + tile_rows - 1) / tile_rows;
                first[e] = low;
                low = next;
            }
            start[c.E] = at;
            first[c.E] = low;
        }
        __syncthreads();
        return;
    }
    int at = incl - mine;
    for (int i = 0; i < warp; ++i) at += sums[i];
    for (int e = e0; e < e1; ++e) {
        start[e] = at;
        at += (max(first[e + 1] - first[e], 0) + tile_rows - 1) / tile_rows;
    }
    if (threadIdx.x == THREADS - 1) start[c.E] = at;
    __syncthreads();
}

__device__ __forceinline__ void put16(uint32_t dst, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// *p, or 0 without looking at it: a predicate, no branch, so that many such loads are in flight at once.
__device__ __forceinline__ uint32_t load_if(const uint16_t* p, bool have) {
    uint16_t v;
    asm("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n mov.u16 %0, 0;\n @q ld.global.nc.u16 %0, [%1];\n}" : "=h"(v) : "l"(p), "r"((int)have));
    return v;
}

// Eight channels of a row that starts on any 2-byte boundary, those from `have` on as zeros.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int have) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = load_if(p + i, i < have);
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

struct Unit {
    int expert, tile;      // tile of output features
    int row0, count;       // rows of y
};

__device__ __forceinline__ int unit_count(const Int4Call& c, int feature_tiles, int tile_rows, const int* start) {
    return feature_tiles * (c.offsets ? start[c.E] : (int)(((int64_t)c.rows + tile_rows - 1) / tile_rows));
}

// Unit u: row tiles of one feature tile are neighbours, so that its weights are read once.
__device__ __forceinline__ Unit unit_at(const Int4Call& c, int u, int feature_tiles, int tile_rows, const int* start,
                                        const int* first) {
    if (!c.offsets) {
        const int tiles = (int)(((int64_t)c.rows + tile_rows - 1) / tile_rows), tile = u / tiles, row0 = (u - tile * tiles) * tile_rows;
        return {0, tile, row0, min(tile_rows, c.rows - row0)};
    }
    const int v = u / feature_tiles;
    int lo = 0, hi = c.E - 1;              // last expert with start[e] <= v
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= v) lo = mid; else hi = mid - 1;
    }
    const int tiles = start[lo + 1] - start[lo], in = u - start[lo] * feature_tiles;
    const int tile = in / tiles, rt = in - tile * tiles;
    const int row0 = first[lo] + rt * tile_rows;
    return {lo, tile, row0, min(tile_rows, first[lo + 1] - row0)};
}

// Row of x that row r of y reads, or -1.
__device__ __forceinline__ int source_row(const Int4Call& c, int r) {
    if (!c.token) return r;
    const int t = c.token[r];
    if (t >= 0 && t < c.x_rows) return t;
    atomicOr(c.status, MOE_DEV_BAD_ROW);
    return -1;
}

// SiLU(g) * u with the correctly rounded quotient: these results may be kept in fp32.  g < -88: exp(-g) is
// infinite and the quotient -0.
__device__ __forceinline__ float gate(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

__device__ __forceinline__ void put_y(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_y(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_y(const Int4Call& c, int row, int n, float v) {
    if (c.y_f32)
        static_cast<float*>(c.y)[row * c.ldy + n] = v;
    else
        static_cast<__nv_bfloat16*>(c.y)[row * c.ldy + n] = __float2bfloat16_rn(v);
}

}  // namespace i4
}  // namespace moe
