// paged_attention.cu -- attention of one new token over a paged key-value cache.
//
// Per sequence b and query head i, with n = seq_lens[b] keys (the last `window` of them where a
// window is given) and kv head h = i / (Hq / Hkv):
//     s_j = scale q . k_j,   m = max_j s_j,   l = sum_j e^(s_j - m),
//     o = sum_j e^(s_j - m) v_j / l,   lse = m + ln l.
// Parts of the keys give (m_i, l_i, a_i = sum e^(s_j - m_i) v_j), which join exactly:
//     m = max m_i,  l = sum e^(m_i - m) l_i,  o = sum e^(m_i - m) a_i / l.
//
// The work is cut into units of UNIT keys of one (sequence, kv head, group of query rows); the
// units of the whole batch are dealt out evenly over the grid, in order, so that one long
// sequence spreads over every SM and a ragged batch stays balanced without the host knowing the
// lengths.  A block whose range ends inside a (sequence, head) writes its part to the workspace;
// a second kernel joins the parts in block order, so that results do not depend on timing.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "paged.cuh"

namespace gret {

namespace {

constexpr int NT = 128;
constexpr int NW = NT / 32;
constexpr int UNIT = 64;       // keys of one unit of work
constexpr int ROWS = 8;        // query rows a block works on at a time
constexpr int GRID = 148 * 4;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// What the join needs of block c: the pair whose first part block c holds (-1: none), and the
// number of blocks that hold parts of it (block c's tail slot, then the head slots of the next).
struct Header {
    int32_t pair, parts;
};

// Parts in the workspace: slot 2c is block c's head (the rest of a pair begun by an earlier
// block), slot 2c + 1 its tail (a pair that a later block goes on with).
template <int D>
struct Part {
    float m[ROWS], l[ROWS];      // m in units of log2
    float a[ROWS][D];
};

struct Params {
    const void* q;
    const int32_t* lens;
    PagedTable table;
    PagedPool pool;
    float scale_log2;
    int window, Hq, G, QG;       // query heads a kv head; groups of ROWS of them
    void* o;
    float* lse;
    int32_t* status;
    Header* headers;
    void* parts;
};

// Keys [first, len) of sequence b.
__device__ __forceinline__ void key_range(const Params& p, int b, int64_t& first, int64_t& len) {
    const int64_t cap = (int64_t)p.table.max_pages << p.pool.page_shift;
    len = p.lens[b];
    if (len < 0 || len > cap) {
        paged_flag(p.status, GRET_PAGED_BAD_LENGTH);
        len = len < 0 ? 0 : cap;
    }
    first = p.window > 0 && len > p.window ? len - p.window : 0;
}

__device__ __forceinline__ int64_t units_of(const Params& p, int b) {
    int64_t first, len;
    key_range(p, b, first, len);
    return (len - first + UNIT - 1) / UNIT;
}

template <typename T, int D>
__global__ void __launch_bounds__(NT) paged_attn_kernel(const Params p) {
    constexpr int E = D / 32;    // dimensions a lane holds
    __shared__ float qs[ROWS][D];
    __shared__ float wm[NW][ROWS], wl[NW][ROWS], wa[NW][ROWS][D];
    __shared__ int64_t scan[NW], start_unit;
    __shared__ int start_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = p.table.S, pairs_b = p.pool.H * p.QG;

    // sequences without keys: zeros
    for (int b = blockIdx.x; b < B; b += gridDim.x)
        if (units_of(p, b) == 0) {
            for (int i = tid; i < p.Hq * D; i += NT)
                static_cast<T*>(p.o)[(int64_t)b * p.Hq * D + i] = from_f32<T>(0.f);
            if (p.lse)
                for (int i = tid; i < p.Hq; i += NT) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
        }

    // this block's range of units, [u0, u1) of U.  With fewer units than blocks, the first U blocks
    // take one each: a pair's parts lie in consecutive blocks
    const int per = (B + NT - 1) / NT;
    int64_t mine = 0;
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) mine += units_of(p, b) * pairs_b;
    int64_t incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t U = 0, before = incl - mine;
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += scan[w];
        U += scan[w];
    }
    const int64_t blocks = min(U, (int64_t)gridDim.x);
    if (blockIdx.x >= blocks) {
        if (tid == 0) p.headers[blockIdx.x] = {-1, 0};
        return;
    }
    const int64_t u0 = U * blockIdx.x / blocks, u1 = U * (blockIdx.x + 1) / blocks;
    if (before <= u0 && u0 < before + mine) {
        int b = tid * per;
        int64_t at = before;
        for (;; ++b) {
            const int64_t x = units_of(p, b) * pairs_b;
            if (u0 < at + x) break;
            at += x;
        }
        start_b = b;
        start_unit = at;
    }
    __syncthreads();
    int b = start_b;
    int64_t first, len;
    key_range(p, b, first, len);
    int64_t nu = (len - first + UNIT - 1) / UNIT;
    int pr = (int)((u0 - start_unit) / nu);              // pair within the sequence
    int64_t t0 = (u0 - start_unit) % nu;                 // first unit of the segment in its pair
    int64_t u = u0;
    Header header = {-1, 0};
    const int page_mask = (1 << p.pool.page_shift) - 1;

    while (u < u1) {
        const int64_t t1 = min(nu, t0 + (u1 - u));
        const int h = pr / p.QG, qg = pr % p.QG;
        const int rows = min(ROWS, p.G - qg * ROWS);
        const int64_t head0 = (int64_t)b * p.Hq + h * p.G + qg * ROWS;   // first query row
        __syncthreads();
        for (int i = tid; i < ROWS * D; i += NT)
            qs[i / D][i % D] = i / D < rows
                                   ? to_f32(static_cast<const T*>(p.q)[head0 * D + i]) * p.scale_log2
                                   : 0.f;
        __syncthreads();
        float m[ROWS], l[ROWS], acc[ROWS][E];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
        }
        const int64_t key1 = min(len, first + t1 * UNIT);
        for (int64_t j = first + t0 * UNIT + warp; j < key1; j += NW) {
            const int id = p.table.entries[b * p.table.stride + (j >> p.pool.page_shift)];
            if ((unsigned)id >= (unsigned)p.pool.n_pages) {
                if (lane == 0) paged_flag(p.status, GRET_PAGED_BAD_PAGE);
                continue;
            }
            const int64_t off = id * p.pool.sp + (j & page_mask) * p.pool.st + h * p.pool.sh;
            const T* kr = reinterpret_cast<const T*>(p.pool.k + off);
            const T* vr = reinterpret_cast<const T*>(p.pool.v + off);
            float kf[E], vf[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                kf[e] = to_f32(kr[lane + 32 * e]);
                vf[e] = to_f32(vr[lane + 32 * e]);
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(qs[r][lane + 32 * e], kf[e], s);
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                const float mn = fmaxf(m[r], s);
                const float base = mn == -INFINITY ? 0.f : mn;
                const float corr = exp2f(m[r] - base), pj = exp2f(s - base);
                l[r] = l[r] * corr + pj;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[r][e] = acc[r][e] * corr + pj * vf[e];
                m[r] = mn;
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (lane == 0) {
                wm[warp][r] = m[r];
                wl[warp][r] = l[r];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) wa[warp][r][lane + 32 * e] = acc[r][e];
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == nu;
        Part<D>* part = static_cast<Part<D>*>(p.parts) + 2 * blockIdx.x + (t0 == 0);
        if (!whole && t0 == 0) {
            // the block that holds unit x is the largest c with floor(c U / blocks) <= x
            const int64_t x = u + nu - 1;
            header.pair = (b * p.pool.H + h) * p.QG + qg;
            header.parts = (int)(((x + 1) * blocks - 1) / U - blockIdx.x) + 1;
        }
        for (int i = tid; i < rows * D; i += NT) {
            const int r = i / D, e = i % D;
            float M = -INFINITY;
            for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w][r]);
            const float base = M == -INFINITY ? 0.f : M;
            float a = 0.f, z = 0.f;
            for (int w = 0; w < NW; ++w) {
                const float f = exp2f(wm[w][r] - base);
                a += wa[w][r][e] * f;
                z += wl[w][r] * f;
            }
            if (whole) {
                static_cast<T*>(p.o)[head0 * D + i] = from_f32<T>(a / z);
                if (p.lse && e == 0) p.lse[head0 + r] = (M + log2f(z)) * LN2;
            } else {
                part->a[r][e] = a;
                if (e == 0) {
                    part->m[r] = M;
                    part->l[r] = z;
                }
            }
        }
        u += t1 - t0;
        t0 = 0;
        if (t1 == nu && ++pr == pairs_b && u < u1) {
            pr = 0;
            do {
                ++b;
                key_range(p, b, first, len);
            } while (len == first);
            nu = (len - first + UNIT - 1) / UNIT;
        }
    }
    if (tid == 0) p.headers[blockIdx.x] = header;
}

// Block c joins the parts of the pair that block c of the kernel above began and did not finish.
template <typename T, int D>
__global__ void __launch_bounds__(NT) paged_join_kernel(const Params p) {
    const Header hd = p.headers[blockIdx.x];
    if (hd.pair < 0) return;
    const int qg = hd.pair % p.QG;
    const int64_t bh = hd.pair / p.QG;
    const int rows = min(ROWS, p.G - qg * ROWS);
    const int64_t head0 = bh * p.G + qg * ROWS;
    const Part<D>* parts = static_cast<const Part<D>*>(p.parts);
    const int c = blockIdx.x;
    for (int i = threadIdx.x; i < rows * D; i += NT) {
        const int r = i / D, e = i % D;
        float M = -INFINITY;
        for (int k = 0; k < hd.parts; ++k) M = fmaxf(M, parts[2 * (c + k) + (k == 0)].m[r]);
        const float base = M == -INFINITY ? 0.f : M;
        float a = 0.f, z = 0.f;
        for (int k = 0; k < hd.parts; ++k) {
            const Part<D>& x = parts[2 * (c + k) + (k == 0)];
            const float f = exp2f(x.m[r] - base);
            a += x.a[r][e] * f;
            z += x.l[r] * f;
        }
        static_cast<T*>(p.o)[head0 * D + i] = from_f32<T>(a / z);
        if (p.lse && e == 0) p.lse[head0 + r] = (M + log2f(z)) * LN2;
    }
}

template <typename T, int D>
cudaError_t launch(const Params& p, cudaStream_t stream) {
    paged_attn_kernel<T, D><<<GRID, NT, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    paged_join_kernel<T, D><<<GRID, NT, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t paged_attn_workspace(bool, int, int, int d) {
    const size_t head = (GRID * sizeof(Header) + 255) / 256 * 256;
    return head + 2 * GRID * (d == 64 ? sizeof(Part<64>) : sizeof(Part<128>));
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
    Params p;
    p.q = a.q;
    p.lens = a.seq_lens;
    p.table = a.table;
    p.pool = a.pool;
    p.scale_log2 = a.scale * LOG2E;
    p.window = a.window;
    p.Hq = a.Hq;
    p.G = a.Hq / a.pool.H;
    p.QG = (p.G + ROWS - 1) / ROWS;
    p.o = a.o;
    p.lse = a.lse;
    p.status = a.status;
    p.headers = static_cast<Header*>(a.workspace);
    p.parts = static_cast<unsigned char*>(a.workspace) + (GRID * sizeof(Header) + 255) / 256 * 256;
    if (a.bf16)
        return a.d == 64 ? launch<__nv_bfloat16, 64>(p, stream)
                         : launch<__nv_bfloat16, 128>(p, stream);
    return a.d == 64 ? launch<float, 64>(p, stream) : launch<float, 128>(p, stream);
}

}  // namespace gret
