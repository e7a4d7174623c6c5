// Tokens sorted by expert (dispatch), the weighted way back (combine) and the
// gradients of both.  All of it moves memory: P pairs of H elements are
// written once (dispatch), read once (combine) or both (combine's gradient),
// and the T tokens' rows once.  Nothing is added by atomics, so every result
// is the same in each run.  8192 tokens x 8 rows x 7168 bf16, against the
// measured copy rate: dispatch 165 us (0.94), combine 161 (0.97), its gradient
// 314 (0.94).
#include <algorithm>

#include "experts_internal.cuh"

namespace moe {

namespace {

__device__ uint32_t g_status;          // MOE_DEV_BAD_ROW, one word per device

constexpr int MAX_K = MOE_DISPATCH_MAX_TOPK;
constexpr int MAX_E = MOE_DISPATCH_MAX_EXPERTS;

// ---------------------------------------------------------------------------
// The sort.  Pair p = t * k + j has key e_p = id - first_expert, "elsewhere"
// when that is not in [0, E), and
//   row(p) = #{p' : e_p' < e_p} + #{p' < p : e_p' = e_p},
// which needs no sorted sequence, only counts.  Up to SMALL_PAIRS pairs every
// CTA counts for the pairs of its own token, over all pairs, one warp per
// pair: 32 comparisons a lane at most, no exchange between CTAs, one launch.
// More pairs are cut into chunks of whole tokens: one kernel counts each
// chunk's pairs per expert, one turns the counts into prefix sums over the
// chunks, and the copying kernel adds its comparisons within the chunk (at
// most SMALL_PAIRS of them) and the totals of the experts below.
// ---------------------------------------------------------------------------
constexpr int SMALL_PAIRS = 1024;
constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr uint32_t ELSEWHERE = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t key_of(int32_t id, int first, int E) {
    const uint32_t e = (uint32_t)id - (uint32_t)first;       // ids below first wrap to 2^31 - E and more
    return e < (uint32_t)E ? e : ELSEWHERE;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

// Exclusive prefix sums of h[0, E) into out[0, E], by the whole CTA.
__device__ void write_offsets(const int* h, int E, int32_t* __restrict__ out) {
    constexpr int PER = MAX_E / THREADS;
    __shared__ int sums[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v[PER], mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x * PER + i;
        v[i] = e < E ? h[e] : 0;
        mine += v[i];
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int i = 0; i < warp; ++i) at += sums[i];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x * PER + i;
        if (e <= E) out[e] = at;
        at += v[i];
    }
    if (threadIdx.x == THREADS - 1 && E == MAX_E) out[E] = at;
}

__global__ void __launch_bounds__(THREADS) count_kernel(const int32_t* __restrict__ ids, int pairs, int chunk_pairs,
                                                        int first, int E, int32_t* __restrict__ cnt) {
    __shared__ int h[MAX_E];
    pdl_trigger();
    for (int e = threadIdx.x; e < E; e += THREADS) h[e] = 0;
    pdl_wait();
    __syncthreads();
    const int p0 = blockIdx.x * chunk_pairs, n = min(chunk_pairs, pairs - p0);
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const uint32_t e = key_of(ids[p0 + i], first, E);
        if (e != ELSEWHERE) atomicAdd(&h[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += THREADS) cnt[(size_t)blockIdx.x * E + e] = h[e];
}

// cnt[c][e] -> sum over c' < c of cnt[c'][e]; cnt[chunks][e] = the expert's
// total.  A CTA has 32 experts, one per lane, and each of its 32 warps a run
// of the chunks.
__global__ void __launch_bounds__(1024) scan_kernel(int32_t* __restrict__ cnt, int chunks, int E) {
    __shared__ int part[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    const int per = (chunks + 31) / 32, c0 = min(chunks, warp * per), c1 = min(chunks, c0 + per);
    int sum = 0;
    if (e < E) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += cnt[(size_t)c * E + e];
    }
    part[warp][lane] = sum;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += part[w][lane];
    if (e >= E) return;
    int32_t* p = cnt + (size_t)c0 * E + e;
    int c = c0;
    for (; c + 8 <= c1; c += 8, p += (size_t)8 * E) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[(size_t)i * E];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[(size_t)i * E] = at;
            at += v[i];
        }
    }
    for (; c < c1; ++c, p += E) {
        const int v = *p;
        *p = at;
        at += v;
    }
    if (warp == 31) *p = at;
}

// ---------------------------------------------------------------------------
// The copy.  A CTA has one token (or, in small batches, a column block of it)
// and holds that part of its row in registers while its warps find the rows
// it goes to; then it stores it once per row.  The last CTA writes the
// offsets.
// ---------------------------------------------------------------------------
enum SortMode { SORT_SMALL, SORT_CHUNKS, SORT_GIVEN };

struct DispatchCall {
    const int32_t* ids;
    int32_t *offsets, *sorted_token, *inv_row;
    const int32_t* base;               // SORT_CHUNKS: [chunks + 1][E] prefix sums, totals last
    const char* x;
    char* rows;
    int64_t ldx, ld_rows;              // bytes
    int T, k, E, first, n_rows, chunk_tokens, chunks;
    int vecs;                          // of a row
    int blocks;                        // column blocks of a row, VECS * THREADS vectors each
};

template <typename V, int VECS, SortMode MODE>
__global__ void __launch_bounds__(THREADS) dispatch_kernel(const DispatchCall c) {
    __shared__ uint32_t keys[SMALL_PAIRS];
    __shared__ int dest[MAX_K + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = c.blocks == 1 ? blockIdx.x : blockIdx.x / c.blocks;
    const int block = c.blocks == 1 ? 0 : blockIdx.x % c.blocks;
    pdl_trigger();
    pdl_wait();
    if (MODE != SORT_GIVEN && t == c.T) {                    // the offsets' CTA
        int* h = reinterpret_cast<int*>(keys);
        if (MODE == SORT_SMALL) {
            for (int e = threadIdx.x; e < c.E; e += THREADS) h[e] = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < c.T * c.k; i += THREADS) {
                const uint32_t e = key_of(c.ids[i], c.first, c.E);
                if (e != ELSEWHERE) atomicAdd(&h[e], 1);
            }
        } else {
            for (int e = threadIdx.x; e < c.E; e += THREADS) h[e] = c.base[(size_t)c.chunks * c.E + e];
        }
        __syncthreads();
        write_offsets(h, c.E, c.offsets);
        return;
    }
    const V* src = reinterpret_cast<const V*>(c.x + t * c.ldx);
    V v[VECS];
    int i0 = block * (VECS * THREADS) + threadIdx.x;
    if (c.x) {
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            if (i0 + i * THREADS < c.vecs) v[i] = src[i0 + i * THREADS];
    }
    const int p0 = t * c.k;
    if (MODE == SORT_GIVEN) {
        if (threadIdx.x < c.k) {
            const int r = c.inv_row[p0 + threadIdx.x];
            const bool ok = r >= 0 && r < c.n_rows;
            if (!ok && r != -1) atomicOr(&g_status, MOE_DEV_BAD_ROW);
            dest[threadIdx.x] = ok ? r : -1;
        }
    } else {
        // this token's keys, and those of the pairs that they are compared with
        int begin = 0, n = c.T * c.k;
        if (MODE == SORT_CHUNKS) {
            begin = t / c.chunk_tokens * c.chunk_tokens * c.k;
            n = p0 + c.k - begin;
        }
        for (int i = threadIdx.x; i < n; i += THREADS) keys[i] = key_of(c.ids[begin + i], c.first, c.E);
        __syncthreads();
        for (int j = warp; j <= c.k; j += WARPS) {           // j = k: how many rows there are
            const int q = p0 + j - begin;
            const uint32_t e = j < c.k ? keys[q] : (uint32_t)c.E;
            int r = -1;
            if (e != ELSEWHERE) {
                int sum = 0;
                if (MODE == SORT_SMALL) {
#pragma unroll 4
                    for (int i = lane; i < n; i += 32) sum += (keys[i] < e) + (i < q && keys[i] == e);
                } else {
                    for (int i = lane; i < (int)e; i += 32) sum += c.base[(size_t)c.chunks * c.E + i];
                    if (j < c.k) {
#pragma unroll 4
                        for (int i = lane; i < q; i += 32) sum += keys[i] == e;
                        if (lane == 0) sum += c.base[(size_t)(t / c.chunk_tokens) * c.E + e];
                    }
                }
                r = warp_sum(sum);
            }
            if (lane == 0) {
                dest[j] = r;
                if (j < c.k && block == 0) {
                    c.inv_row[p0 + j] = r;
                    if (r >= 0) c.sorted_token[r] = t;
                    if (c.x && r >= c.n_rows) atomicOr(&g_status, MOE_DEV_BAD_ROW);
                }
            }
        }
    }
    __syncthreads();
    if (MODE != SORT_GIVEN && block == 0 && threadIdx.x < c.k && p0 + (int)threadIdx.x >= dest[c.k])
        c.sorted_token[p0 + threadIdx.x] = -1;
    if (!c.x) return;
    while (true) {
        for (int j = 0; j < c.k; ++j) {
            const int r = dest[j];
            if (r < 0 || r >= c.n_rows) continue;
            V* dst = reinterpret_cast<V*>(c.rows + r * c.ld_rows);
#pragma unroll
            for (int i = 0; i < VECS; ++i)
                if (i0 + i * THREADS < c.vecs) dst[i0 + i * THREADS] = v[i];
        }
        i0 += c.blocks * (VECS * THREADS);
        if (i0 >= c.vecs) return;
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            if (i0 + i * THREADS < c.vecs) v[i] = src[i0 + i * THREADS];
    }
}

template <typename V>
cudaError_t launch_copy(DispatchCall& c, bool given, int row_bytes, cudaStream_t s) {
    constexpr int VECS = 4;
    c.vecs = c.x ? row_bytes / (int)sizeof(V) : 0;
    c.blocks = 1;
    if (given) {
        return launch_pdl(dispatch_kernel<V, VECS, SORT_GIVEN>, dim3(c.T), dim3(THREADS), 0, s, c);
    }
    if (c.chunks) return launch_pdl(dispatch_kernel<V, VECS, SORT_CHUNKS>, dim3(c.T + 1), dim3(THREADS), 0, s, c);
    // few tokens: a row over as many CTAs as give every thread one vector
    c.blocks = std::max(1, std::min(64, (c.vecs + THREADS - 1) / THREADS));
    return launch_pdl(dispatch_kernel<V, 1, SORT_SMALL>, dim3(c.T * c.blocks + 1), dim3(THREADS), 0, s, c);
}

// ---------------------------------------------------------------------------
// Combine: a thread has 8 columns of one token and loads them from 8 rows (fp32: 4) at a time before it adds
// them up.  Rows off the 16-byte grid: four single columns, C_THREADS apart, of 8 rows.
// ---------------------------------------------------------------------------
constexpr int C_THREADS = 128;
constexpr int c_parts(int n) { return n == 1 ? 4 : 1; }

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// N consecutive elements as they lie in memory: 8 in 16-byte words, or 1.
template <typename T, int N>
struct Pack {
    uint4 w[N * sizeof(T) / 16];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        if (sizeof(T) == 4) return __uint_as_float(u[i]);
        return __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
    }
    __device__ __forceinline__ void set2(int i, float a, float b) {      // elements i, i + 1 (i even)
        uint32_t* u = reinterpret_cast<uint32_t*>(w);
        if (sizeof(T) == 4) {
            u[i] = __float_as_uint(a);
            u[i + 1] = __float_as_uint(b);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            u[i >> 1] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
};
template <typename T>
struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
};
template <typename T>
__device__ __forceinline__ void put(Pack<T, 8>& p, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) p.set2(i, f[i], f[i + 1]);
}
template <typename T>
__device__ __forceinline__ void put(Pack<T, 1>& p, const float (&f)[1]) { p.v = from_f32<T>(f[0]); }

// This thread's slot of the token: its row, or -1 where there is none.
__device__ __forceinline__ int checked_row(int r, int n_rows) {
    const bool ok = r >= 0 && r < n_rows;
    if (!ok && r != -1) atomicOr(&g_status, MOE_DEV_BAD_ROW);
    return ok ? r : -1;
}

template <typename TO, typename TY, int N>
__global__ void __launch_bounds__(C_THREADS) combine_rows_kernel(const moe_combine_args a) {
    __shared__ int row[MAX_K];
    __shared__ float wt[MAX_K];
    const int64_t t = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    pdl_trigger();
    pdl_wait();
    if (t >= a.tokens) return;
    const int k = a.top_k;
    if (threadIdx.x < k) {
        row[threadIdx.x] = checked_row(a.inv_row[t * k + threadIdx.x], a.n_rows);
        wt[threadIdx.x] = a.w ? a.w[t * k + threadIdx.x] : 1.0f;
    }
    __syncthreads();
    constexpr int C = c_parts(N), STEP = C_THREADS * N;      // parts of a thread, so many columns apart
    const int col = (blockIdx.x * C * C_THREADS + threadIdx.x) * N;
    if (col >= a.cols) return;
    const TO* o = static_cast<const TO*>(a.o) + col;
    float acc[C][N];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        Pack<TY, N> v;
        const bool have = a.add && col + c * STEP < a.cols;
        if (have) v.load(static_cast<const TY*>(a.add) + t * a.ld_add + col + c * STEP);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[c][i] = have ? v.get(i) : 0.f;
    }
    constexpr int J = N == 1 || sizeof(TO) == 2 ? 8 : 4;
    for (int j0 = 0; j0 < k; j0 += J) {
        Pack<TO, N> v[J][C];
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (j0 + j < k && row[j0 + j] >= 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (col + c * STEP < a.cols) v[j][c].load(o + row[j0 + j] * a.ldo + c * STEP);
            }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (j0 + j < k && row[j0 + j] >= 0) {
                const float w = wt[j0 + j];
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[c][i] = __fmaf_rn(w, v[j][c].get(i), acc[c][i]);
            }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (col + c * STEP < a.cols) {
            Pack<TY, N> out;
            put(out, acc[c]);
            out.store(static_cast<TY*>(a.y) + t * a.ldy + col + c * STEP);
        }
}

// ---------------------------------------------------------------------------
// Combine's gradient.  A CTA has one token (few tokens: one slot of it), its
// threads hold VECS pieces of dy and go over the rows: load o, store w * dy,
// add up the products.  The sums meet by shuffles, then over the warps in
// order.
// ---------------------------------------------------------------------------
template <typename TO, typename TY, int N>
__global__ void __launch_bounds__(THREADS) combine_grad_kernel(const moe_combine_grad_args a) {
    constexpr int VECS = 4;
    __shared__ int row[MAX_K];
    __shared__ float wt[MAX_K];
    __shared__ float sums[MAX_K][WARPS];
    const int t = blockIdx.x, k = a.top_k;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int jstep = gridDim.y;
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < k) {
        row[threadIdx.x] = checked_row(a.inv_row[(int64_t)t * k + threadIdx.x], a.n_rows);
        wt[threadIdx.x] = a.w ? a.w[(int64_t)t * k + threadIdx.x] : 1.0f;
    }
    for (int i = threadIdx.x; i < MAX_K * WARPS; i += THREADS) (&sums[0][0])[i] = 0.f;
    __syncthreads();
    const TY* dy = static_cast<const TY*>(a.dy) + t * a.ld_dy;
    for (int col0 = threadIdx.x * N; col0 < (a.cols + THREADS * N - 1) / (THREADS * N) * (THREADS * N);
         col0 += VECS * THREADS * N) {
        Pack<TY, N> g[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            if (col0 + i * THREADS * N < a.cols) g[i].load(dy + col0 + i * THREADS * N);
        for (int j = blockIdx.y; j < k; j += jstep) {
            const int r = row[j];
            if (r < 0) continue;
            Pack<TO, N> v[VECS];
            if (a.d_w) {
                const TO* o = static_cast<const TO*>(a.o) + r * a.ldo;
#pragma unroll
                for (int i = 0; i < VECS; ++i)
                    if (col0 + i * THREADS * N < a.cols) v[i].load(o + col0 + i * THREADS * N);
            }
            if (a.d_o) {
                TO* d = static_cast<TO*>(a.d_o) + r * a.ld_d_o;
                const float w = wt[j];
#pragma unroll
                for (int i = 0; i < VECS; ++i)
                    if (col0 + i * THREADS * N < a.cols) {
                        float f[N];
#pragma unroll
                        for (int e = 0; e < N; ++e) f[e] = w * g[i].get(e);
                        Pack<TO, N> out;
                        put(out, f);
                        out.store(d + col0 + i * THREADS * N);
                    }
            }
            if (a.d_w) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < VECS; ++i)
                    if (col0 + i * THREADS * N < a.cols) {
#pragma unroll
                        for (int e = 0; e < N; ++e) sum = __fmaf_rn(v[i].get(e), g[i].get(e), sum);
                    }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
                if (lane == 0) sums[j][warp] += sum;
            }
        }
    }
    if (!a.d_w) return;
    __syncthreads();
    const int j = blockIdx.y + threadIdx.x * jstep;
    if (j < k) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) sum += sums[j][w];
        a.d_w[(int64_t)t * k + j] = sum;
    }
}

// Whether rows from p on, ld elements of `size` bytes apart, lie on `to`-byte boundaries.
bool on_grid(const void* p, int64_t ld, int size, int to) {
    return !p || (reinterpret_cast<uintptr_t>(p) % to == 0 && ld * size % to == 0);
}

int size_of(int type) { return type == MOE_F32 ? 4 : 2; }

}  // namespace

cudaError_t dispatch_status_word(uint32_t** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_status); }

SortPlan plan_sort(int tokens, int top_k) {
    // chunks of at least 64 pairs and at most SMALL_PAIRS, 256 of them where that lies between
    const int least = (64 + top_k - 1) / top_k, most = SMALL_PAIRS / top_k;
    if ((int64_t)tokens * top_k <= SMALL_PAIRS) return {tokens, 0, 0};
    const int chunk = std::min(most, std::max((tokens - 1) / 256 + 1, least));
    return {chunk, (tokens - 1) / chunk + 1, std::max(std::min(256, (tokens - 1) / least + 1), (tokens - 1) / most + 1)};
}

cudaError_t launch_dispatch(const moe_dispatch_args* a, int32_t* ws, cudaStream_t s) {
    DispatchCall c = {};
    c.ids = a->ids;
    c.offsets = a->expert_offsets;
    c.sorted_token = a->sorted_token;
    c.inv_row = a->inv_row;
    c.base = ws;
    const int size = size_of(a->x_type), row_bytes = a->cols * size;
    c.x = static_cast<const char*>(a->x);
    c.rows = static_cast<char*>(a->rows);
    c.ldx = a->ldx * size;
    c.ld_rows = a->ld_rows * size;
    c.T = a->tokens;
    c.k = a->top_k;
    c.E = a->n_experts;
    c.first = a->first_expert;
    c.n_rows = a->n_rows;
    if (a->ids) {
        const SortPlan plan = plan_sort(a->tokens, a->top_k);
        c.chunk_tokens = plan.chunk_tokens;
        c.chunks = plan.chunks;
        if (plan.chunks) {
            cudaError_t e = launch_pdl(count_kernel, dim3(plan.chunks), dim3(THREADS), 0, s, a->ids, a->tokens * a->top_k,
                                       plan.chunk_tokens * a->top_k, a->first_expert, a->n_experts, ws);
            if (e != cudaSuccess) return e;
            e = launch_pdl(scan_kernel, dim3((a->n_experts + 31) / 32), dim3(1024), 0, s, ws, plan.chunks, a->n_experts);
            if (e != cudaSuccess) return e;
        }
    }
    auto fits = [&](int to) {
        return row_bytes % to == 0 && on_grid(a->x, a->ldx, size, to) && on_grid(a->rows, a->ld_rows, size, to);
    };
    if (fits(16)) return launch_copy<uint4>(c, !a->ids, row_bytes, s);
    if (fits(4)) return launch_copy<uint32_t>(c, !a->ids, row_bytes, s);
    return launch_copy<uint16_t>(c, !a->ids, row_bytes, s);
}

namespace {

template <typename TO, typename TY>
cudaError_t combine_typed(const moe_combine_args* a, bool vec, cudaStream_t s) {
    const int cols = C_THREADS * (vec ? 8 : c_parts(1));
    const dim3 grid((a->cols + cols - 1) / cols, std::min(a->tokens, 32768), (a->tokens - 1) / 32768 + 1);
    return vec ? launch_pdl(combine_rows_kernel<TO, TY, 8>, grid, dim3(C_THREADS), 0, s, *a)
               : launch_pdl(combine_rows_kernel<TO, TY, 1>, grid, dim3(C_THREADS), 0, s, *a);
}

template <typename TO, typename TY>
cudaError_t grad_typed(const moe_combine_grad_args* a, bool vec, cudaStream_t s) {
    // a slot per CTA while that fills the GPU no more than once
    const dim3 grid(a->tokens, (int64_t)a->tokens * a->top_k <= 1024 ? a->top_k : 1);
    return vec ? launch_pdl(combine_grad_kernel<TO, TY, 8>, grid, dim3(THREADS), 0, s, *a)
               : launch_pdl(combine_grad_kernel<TO, TY, 1>, grid, dim3(THREADS), 0, s, *a);
}

}  // namespace

cudaError_t launch_combine_rows(const moe_combine_args* a, cudaStream_t s) {
    const bool of = a->o_type == MOE_F32, yf = a->y_type == MOE_F32;
    const int os = size_of(a->o_type), ys = size_of(a->y_type);
    const bool vec = a->cols % 8 == 0 && on_grid(a->o, a->ldo, os, 16) && on_grid(a->add, a->ld_add, ys, 16) &&
                     on_grid(a->y, a->ldy, ys, 16);
    if (of) return yf ? combine_typed<float, float>(a, vec, s) : combine_typed<float, __nv_bfloat16>(a, vec, s);
    return yf ? combine_typed<__nv_bfloat16, float>(a, vec, s) : combine_typed<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
}

cudaError_t launch_combine_grad(const moe_combine_grad_args* a, cudaStream_t s) {
    const bool of = a->o_type == MOE_F32, yf = a->y_type == MOE_F32;
    const int os = size_of(a->o_type), ys = size_of(a->y_type);
    const bool vec = a->cols % 8 == 0 && on_grid(a->dy, a->ld_dy, ys, 16) && on_grid(a->d_w ? a->o : nullptr, a->ldo, os, 16) &&
                     on_grid(a->d_o, a->ld_d_o, os, 16);
    if (of) return yf ? grad_typed<float, float>(a, vec, s) : grad_typed<float, __nv_bfloat16>(a, vec, s);
    return yf ? grad_typed<__nv_bfloat16, float>(a, vec, s) : grad_typed<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
}

}  // namespace moe
