// Products with 4-bit weights, few rows per matrix, and the repack of the
// weights.
//
// The weights are streamed once and bound the call: half a byte and its share
// of a scale per weight.  At 6.8 TB/s that is 47 weights a clock on each SM,
// so what is done per weight has to stay small.  The codes go from memory into
// each lane's own slots of a ring in shared memory (16 bytes a copy, no lane
// waits for another's codes), are widened by a mask and a subtraction per
// pair, and enter mma.sync.m16n8k16 as the 16-row operand with 8 rows of x as
// the other.  That path gives 1024 products a clock and SM (measured), 128
// weights at 8 rows and 64 at 16: enough for the stream, without the trip of
// every weight through shared memory that tcgen05 operands would need.
//
// A unit is RB blocks of 16 weight rows and NB * 8 rows of x.  The warps of a
// CTA share its input channels, so that each reads its own part of x and of
// the weights; their sums meet in shared memory in the order of the warps.
// CTAs are persistent; the ring is filled for the next unit while one ends.
#include <algorithm>

#include "int4.cuh"

namespace moe {

namespace {

constexpr int THREADS = 256, WARPS = 8;

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One warp's slot of the ring: a tile of RB blocks and of NB * 8 rows of x.
template <int RB, int NB, int SUB>
struct Slot {
    uint4 w[RB][32];
    uint2 x[NB][4][32];                // [channels 16 i + 4 q][lane]
    uint2 s[SUB][RB][8];               // pairs (row g, row g + 8): two fp32, or two bf16 in .x
    uint32_t z[SUB][RB][8];
};

template <int RB, int NB, int SUB, int DEPTH>
struct Smem {
    Slot<RB, NB, SUB> ring[WARPS][DEPTH];
    float sums[WARPS][NB * 8][RB * I4_ROWS + 4];      // + 4: the lanes' rows fall into different banks
    int table[1];                      // start[E + 1], first[E + 1]
};

// SUB: scales per tile and row (2 where a group may end inside a tile).
template <int RB, int NB, int SUB, int DEPTH>
__global__ void __launch_bounds__(THREADS) int4_few_kernel(const Int4Call c) {
    extern __shared__ __align__(16) char smem_raw[];
    auto& sm = *reinterpret_cast<Smem<RB, NB, SUB, DEPTH>*>(smem_raw);
    int* start = sm.table;
    int* first = sm.table + c.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int feature_tiles = c.blocks / RB;
    // this warp's tiles of 64 channels
    const int per = (c.kt + WARPS - 1) / WARPS, t0 = min(c.kt, warp * per), steps = min(c.kt, t0 + per) - t0;
    pdl_trigger();
    pdl_wait();
    i4::row_tiles<THREADS>(c, NB * 8, start, first);
    const int units = start[c.E] * feature_tiles;

    // what is copied next
    int p_unit = blockIdx.x, p_step = 0, p_slot = 0;
    const uint4* p_w = nullptr;
    size_t p_rec = 0;
    int64_t p_x[NB];
    auto enter = [&](int u) {
        const i4::Unit un = i4::unit_at(c, u, feature_tiles, NB * 8, start, first);
        const size_t block = (size_t)un.expert * c.blocks + un.tile * RB;
        p_w = c.w + (block * c.kt + t0) * 32 + lane;
        p_rec = (block + (lane >> 3)) * c.groups * 8 + (lane & 7);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int m = n * 8 + g;
            const int r = m < un.count ? i4::source_row(c, un.row0 + m) : -1;
            p_x[n] = r < 0 ? -1 : r * c.ldx;
        }
    };
    auto copy_next = [&]() {
        if (p_unit < units) {
            Slot<RB, NB, SUB>& slot = sm.ring[warp][p_slot];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) i4::copy16(smem_addr(&slot.w[rb][lane]), p_w + (size_t)rb * c.kt * 32);
            const int t = t0 + p_step;
            if (lane < RB * 8) {
#pragma unroll
                for (int sub = 0; sub < SUB; ++sub) {
                    const size_t rec = p_rec + (size_t)i4::group_of(c, 2 * t + sub) * 8;
                    const uint32_t to = smem_addr(&slot.s[sub][lane >> 3][lane & 7]);
                    if (c.s_f32) i4::copy_small<8>(to, c.s + rec * 8);
                    else i4::copy_small<4>(to, c.s + rec * 4);
                    if (c.z) i4::copy_small<4>(smem_addr(&slot.z[sub][lane >> 3][lane & 7]), c.z + rec);
                }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = t * I4_K + i * 16 + q * 4;
                    const int have = p_x[n] < 0 ? 0 : min(max(c.K - k, 0), 4);
                    const uint16_t* src = have ? c.x + p_x[n] + k : c.x;
                    if (c.x_grid >= 8) {
                        i4::copy8(smem_addr(&slot.x[n][i][lane]), src, have * 2);
                    } else {
                        uint16_t* to = reinterpret_cast<uint16_t*>(&slot.x[n][i][lane]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) to[j] = j < have ? src[j] : (uint16_t)0;
                    }
                }
            }
            p_w += 32;
            if (++p_step == steps) {
                p_step = 0;
                p_unit += gridDim.x;
                if (p_unit < units) enter(p_unit);
            }
        }
        p_slot = p_slot + 1 == DEPTH ? 0 : p_slot + 1;
        i4::copy_commit();
    };

    if (steps > 0) {
        if (p_unit < units) enter(p_unit);
#pragma unroll
        for (int i = 0; i < DEPTH - 1; ++i) copy_next();
    }
    int slot_at = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        float acc[RB][NB][4];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[rb][n][i] = 0.f;
        for (int step = 0; step < steps; ++step) {
            i4::copy_wait<DEPTH - 2>();
            __syncwarp();                      // the other lanes' copies (scales), and their reads of the slot filled next
            copy_next();
            const Slot<RB, NB, SUB>& slot = sm.ring[warp][slot_at];
            slot_at = slot_at + 1 == DEPTH ? 0 : slot_at + 1;
            uint2 xv[NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[n][i] = slot.x[n][i][lane];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const uint4 w = slot.w[rb][lane];
                float part[NB][4];
#pragma unroll
                for (int half = 0; half < 2; ++half) {         // 32 channels: two k16 steps
                    const int sub = SUB == 2 ? half : 0;
                    const uint32_t zp = c.z ? slot.z[sub][rb][g] : I4_ZERO;
                    uint32_t lo[4], hi[4];
                    i4::widen(half ? w.y : w.x, __byte_perm(zp, 0, 0x1010), lo);
                    i4::widen(half ? w.w : w.z, __byte_perm(zp, 0, 0x3232), hi);
                    if (half == 0 || SUB == 2) {
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
                    }
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        mma(part[n], a0, xv[n][2 * half].x, xv[n][2 * half].y);
                        mma(part[n], a1, xv[n][2 * half + 1].x, xv[n][2 * half + 1].y);
                    }
                    if (half == 1 || SUB == 2) {
                        const uint2 sv = slot.s[sub][rb][g];
                        const float s0 = c.s_f32 ? __uint_as_float(sv.x) : __uint_as_float(sv.x << 16);
                        const float s1 = c.s_f32 ? __uint_as_float(sv.y) : __uint_as_float(sv.x & 0xFFFF0000u);
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            acc[rb][n][0] = __fmaf_rn(s0, part[n][0], acc[rb][n][0]);
                            acc[rb][n][1] = __fmaf_rn(s0, part[n][1], acc[rb][n][1]);
                            acc[rb][n][2] = __fmaf_rn(s1, part[n][2], acc[rb][n][2]);
                            acc[rb][n][3] = __fmaf_rn(s1, part[n][3], acc[rb][n][3]);
                        }
                    }
                }
            }
        }
        const i4::Unit un = i4::unit_at(c, u, feature_tiles, NB * 8, start, first);
        float(*mine)[RB * I4_ROWS + 4] = sm.sums[warp];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                mine[n * 8 + 2 * q][rb * 16 + g] = acc[rb][n][0];
                mine[n * 8 + 2 * q + 1][rb * 16 + g] = acc[rb][n][1];
                mine[n * 8 + 2 * q][rb * 16 + g + 8] = acc[rb][n][2];
                mine[n * 8 + 2 * q + 1][rb * 16 + g + 8] = acc[rb][n][3];
            }
        __syncthreads();
        const int wide = c.gated ? RB * 8 : RB * 16;           // output features of a tile
        for (int i = threadIdx.x; i < un.count * wide; i += THREADS) {
            const int m = i / wide, f = i - m * wide;
            const int n = un.tile * wide + f;
            if (n >= c.N) continue;
            if (c.gated) {
                const int at = (f >> 3) * 16 + (f & 7);
                float gate = 0.f, up = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    gate += sm.sums[w][m][at];
                    up += sm.sums[w][m][at + 8];
                }
                i4::store_y(c, un.row0 + m, n, i4::gate(gate, up));
            } else {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) sum += sm.sums[w][m][f];
                i4::store_y(c, un.row0 + m, n, sum);
            }
        }
        __syncthreads();
    }
    i4::copy_wait<0>();
}

template <int RB, int NB, int SUB>
cudaError_t launch(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    constexpr int DEPTH = RB == 4 ? 3 : 4;
    constexpr auto kernel = int4_few_kernel<RB, NB, SUB, DEPTH>;
    const int bytes = sizeof(Smem<RB, NB, SUB, DEPTH>) + 2 * (c.E + 1) * (int)sizeof(int);
    constexpr int most = sizeof(Smem<RB, NB, SUB, DEPTH>) + 2 * (MOE_DISPATCH_MAX_EXPERTS + 1) * (int)sizeof(int);
    static_assert(most <= 227 * 1024, "shared memory");
    cudaError_t e = ensure_smem_limit<kernel>(most);
    if (e != cudaSuccess) return e;
    const int per_sm = std::min(4, 227 * 1024 / (bytes + 1024));
    const int64_t tiles = c.blocks / RB;
    // with offsets no more row tiles than full ones and one for each expert
    const int64_t row_tiles = c.offsets ? std::min<int64_t>(c.rows, c.rows / (NB * 8) + c.E) : (c.rows + NB * 8 - 1) / (NB * 8);
    const int64_t grid = std::min<int64_t>(tiles * row_tiles, (int64_t)L->num_sms * per_sm);
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(THREADS), bytes, s, c);
}

template <int RB, int NB>
cudaError_t launch_sub(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    return L->d.group % I4_K ? launch<RB, NB, 2>(L, c, s) : launch<RB, NB, 1>(L, c, s);
}

template <int RB>
cudaError_t launch_rows(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    const int64_t rows = c.offsets ? (int64_t)c.rows / c.E * 4 : c.rows;
    if (rows <= 8) return launch_sub<RB, 1>(L, c, s);
    if (rows <= 16) return launch_sub<RB, 2>(L, c, s);
    return launch_sub<RB == 4 ? 2 : RB, 4>(L, c, s);
}

// One thread per lane's 16 bytes.
__global__ void __launch_bounds__(256) int4_repack_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ q_up,
                                                          int N, int K, int blocks, int kt, int64_t total,
                                                          uint4* __restrict__ w) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int lane = i & 31, g = lane >> 2, qd = lane & 3;
        const int64_t tile = i >> 5;
        const int t = tile % kt;
        const int64_t eb = tile / kt;
        const int block = eb % blocks;
        const int64_t e = eb / blocks;
        const int64_t row_bytes = (K + 1) / 2;
        uint32_t out[4] = {};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int n = q_up ? block * 8 + g : block * 16 + g + 8 * r;
            if (n >= N) continue;
            const uint8_t* src = (q_up && r ? q_up : q) + (e * N + n) * row_bytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int at = (t * I4_K + h * 32 + (b >> 1) * 16 + qd * 4 + (b & 1) * 2) / 2;
                    const uint32_t byte = at < row_bytes ? src[at] : 0u;
                    v |= (byte & 15u) << (4 * b) | (byte >> 4) << (16 + 4 * b);
                }
                out[r * 2 + h] = v;
            }
        }
        w[i] = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

// One thread per pair of scales.
template <typename T>
__global__ void __launch_bounds__(256) int4_scales_kernel(const T* __restrict__ s, const T* __restrict__ s_up,
                                                          const uint8_t* __restrict__ z, const uint8_t* __restrict__ z_up,
                                                          int N, int src_groups, int blocks, int groups, int64_t total,
                                                          T* __restrict__ s_out, uint32_t* __restrict__ z_out) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int g = i & 7;
        const int64_t rec = i >> 3;
        const int gi = rec % groups;
        const int64_t eb = rec / groups;
        const int block = eb % blocks;
        const int64_t e = eb / blocks;
        uint32_t zs[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int n = s_up ? block * 8 + g : block * 16 + g + 8 * r;
            const bool have = n < N && gi < src_groups;
            const int64_t at = (e * N + n) * src_groups + gi;
            s_out[2 * i + r] = have ? (s_up && r ? s_up : s)[at] : T(0.f);
            zs[r] = have && z ? (z_up && r ? z_up : z)[at] & 127u : 8u;
        }
        if (z_out) z_out[i] = 0x43004300u | zs[0] | zs[1] << 16;
    }
}

}  // namespace

cudaError_t launch_int4_repack(const moe_int4* L, const moe_int4_weights* w, cudaStream_t s) {
    const moe_int4_desc& d = L->d;
    const int64_t words = (int64_t)d.n_experts * L->blocks * L->kt * 32;
    const int64_t recs = (int64_t)d.n_experts * L->blocks * L->groups * 8;
    auto grid = [](int64_t n) { return dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20)); };
    int4_repack_kernel<<<grid(words), 256, 0, s>>>(w->q, d.gated ? w->q_up : nullptr, d.out_features, d.in_features, L->blocks, L->kt,
                                                   words, L->w);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int src_groups = (d.in_features - 1) / d.group + 1;
    const uint8_t* z_up = d.gated ? w->z_up : nullptr;
    if (d.scale_type == MOE_F32)
        int4_scales_kernel<<<grid(recs), 256, 0, s>>>(static_cast<const float*>(w->s), static_cast<const float*>(d.gated ? w->s_up : nullptr),
                                                      w->z, z_up, d.out_features, src_groups, L->blocks, L->groups, recs,
                                                      static_cast<float*>(L->s), L->z);
    else
        int4_scales_kernel<<<grid(recs), 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w->s),
                                                      static_cast<const __nv_bfloat16*>(d.gated ? w->s_up : nullptr), w->z, z_up,
                                                      d.out_features, src_groups, L->blocks, L->groups, recs,
                                                      static_cast<__nv_bfloat16*>(L->s), L->z);
    return cudaGetLastError();
}

cudaError_t launch_int4_few(const moe_int4* L, const Int4Call& c, cudaStream_t s) {
    const int64_t blocks = (int64_t)c.blocks * (c.offsets ? std::min(c.E, c.rows) : 1);
    if (blocks <= 4 * L->num_sms) return launch_rows<1>(L, c, s);
    return launch_rows<4>(L, c, s);
}

}  // namespace moe
